"""The 4-bit cache and the answers' log probabilities as a serving loop uses them:
with the page map, the acceptance and the commit, at once on two streams, and
captured in several waves."""
import pytest
import torch

import kv4_ref as ref
import kvq_ref
import speculative_decoding_diffusion_gb300 as pkg
from speculative_decoding_diffusion_gb300 import binding
from test_gpu_kv4 import ORDER, case, check_keys, close, cu_of, i32, make_cache, put, tables, verify, workspace
from test_gpu_logprobs import near

pytestmark = pytest.mark.gpu
PAGE = 16


def test_steps_of_the_loop():
    """Requests admitted, their prompts appended; twice a pass: attention, logits, the greedy walk, the commit, the closed
    blocks' tokens appended, log probabilities of what was decided; every stage fed by the one before."""
    g = torch.Generator().manual_seed(40)
    Hq, Hkv, hd, B, batch, width, cap, vocab = 4, 2, 128, 4, 3, 8, 30, 3001
    spec = dict(base=1e4, rotary_dim=64)
    lens0 = [37, 5, 64]
    free, queue = i32(torch.randperm(cap, generator=g)), i32([0, cap])
    table, held, served = i32(torch.zeros(batch, width)), i32([0] * batch), i32([0] * batch)
    ws_map, ws_acc, ws_lp = workspace(), None, None
    state = make_cache(g, cap, Hkv, hd)
    dev = state.cuda()
    head = (torch.randn(Hq * hd, vocab, generator=g) * 0.3).cuda()

    def append(k, v, start, n, take=None):
        nonlocal state
        put(k.cuda(), v.cuda(), start, n, table.cpu(), dev, spec, take)
        cu = cu_of(n)
        pos = torch.cat([torch.arange(s, s + m) for s, m in zip(start, n)])
        x = kvq_ref.rope(k, pos, spec)
        t = table.cpu()
        want = ref.append(ref.append(state, 1, v.double(), start, cu, t, take), 0, x, start, cu, t, take)
        got = dev.cpu()
        assert torch.equal(got[..., 8 * hd:16 * hd], want[..., 8 * hd:16 * hd]) and torch.equal(got[..., 17 * hd:], want[..., 17 * hd:])
        kept = torch.cat([torch.arange(int(cu[b]), int(cu[b]) + (n[b] if take is None else take[b])) for b in range(len(n))])
        seq = torch.repeat_interleave(torch.arange(len(n)), torch.tensor(n))
        slots = [(int(t[seq[r], pos[r] // PAGE]), int(pos[r] % PAGE)) for r in kept.tolist()]
        if slots:
            check_keys(got, want, x[kept], slots)
        state = got

    pkg.page_map(i32(lens0), None, held, queue, free, table, held, queue, served, None, ws_map, 0)
    assert served.tolist() == [1, 1, 1]
    N = sum(lens0)
    append(torch.randn(N, Hkv, hd, generator=g).bfloat16(), torch.randn(N, Hkv, hd, generator=g).bfloat16(), [0] * batch, lens0)
    cu = cu_of([B] * batch)
    lens, decided = i32(lens0), i32([0] * batch)
    tokens = torch.randint(0, vocab, (B * batch,), generator=g, dtype=torch.int32).cuda()
    tau = torch.cat([torch.randperm(B, generator=g) + 1 for _ in range(batch)])
    done = i32([0] * batch)
    for step in range(3):
        L = lens.tolist()
        q, kn, vn = (torch.randn(2 * B * batch, h, hd, generator=g).bfloat16() for h in (Hq, Hkv, Hkv))
        out, ws = verify(q.cuda(), dev, table.cpu(), kn.cuda(), vn.cuda(), i32(tau), L, cu, B, spec, 0.09, "paired")
        assert pkg.read_status(ws) == 0
        want, off = ref.verify(q, state, table.cpu().long(), kn, vn, tau, L, cu, spec, 0.09, "paired", 0, 2.0 ** -11)
        close(out, want, off, "bf16")
        # the mask slots' rows, one for each position of the block
        rows = torch.cat([torch.arange(B) + 2 * B * b + B for b in range(batch)]).cuda()
        logits = (out[rows].float().flatten(1) @ head).bfloat16()
        best = logits.float().argmax(-1).int()
        tokens = torch.where((torch.arange(B * batch, device="cuda") % (3 + step)) > 0, best, tokens) if step < 2 else best
        n_acc, tok, pos = (i32([0] * batch) for _ in range(3))
        args = (logits, None, tokens, i32(tau), i32(cu), None, n_acc, tok, pos)
        if ws_acc is None:
            ws_acc = workspace(1 << 16)
        pkg.accept(*args, ws_acc, B * batch, B, rule=binding.SIMSD_ACCEPT_GREEDY, decided=decided)
        binding.commit(i32(cu), i32(tau), n_acc, tok, pos, tokens, decided, lens, done, ws_acc, B * batch, B)
        # what is decided by now gets its log probability; the rest is left out
        ask = torch.where(i32(tau) <= torch.where(done > 0, B, decided).repeat_interleave(B), tokens, -1)
        lp, ent = (torch.full((B * batch,), 7.0, device="cuda") for _ in range(2))
        rank = torch.full((B * batch,), 7, dtype=torch.int32, device="cuda")
        ids, top = torch.full((B * batch, 3), 7, dtype=torch.int32, device="cuda"), torch.full((B * batch, 3), 7.0, device="cuda")
        a = (logits, ask.int(), lp, rank, ent, ids, top)
        if ws_lp is None:
            ws_lp = workspace(pkg.token_logprobs_workspace_size(*a))
        pkg.token_logprobs(*a, ws_lp)
        want_lp = torch.log_softmax(logits.double().cpu(), -1)
        on = (ask >= 0).cpu()
        near(lp.cpu()[on], want_lp.gather(1, tokens.cpu().long()[:, None])[:, 0][on])
        assert (lp.cpu()[~on] == 7).all() and (ids.cpu()[~on] == 7).all()
        assert torch.equal(ids[:, 0].cpu()[on], best.cpu()[on])
        # closed blocks: their data section's tokens stay in the cache
        keep = [B if d else 0 for d in done.tolist()]
        pkg.page_map(i32(L), i32(cu_of(keep)), held, queue, free, table, held, queue, served, None, ws_map, 2 * B * batch)
        assert served.tolist() == [1] * batch
        append(kn, vn, L, [2 * B] * batch, keep)
        assert lens.tolist() == [x + m for x, m in zip(L, keep)]
    assert pkg.read_status(ws_map) == 0 and pkg.read_status(ws_lp) == 0
    assert sum(lens.tolist()) > sum(lens0)


@pytest.mark.parametrize("B", [1, 16])
def test_two_streams_at_once(B):
    """Calls on two streams with workspaces of their own, over the same pages, equal the same calls one after another."""
    lens = (3000, 700, 41)
    cache, table, cu, q, kn, vn, tau = case(B, lens, [B] * 3, "causal", "bf16", 4, 2, 128)
    spec = dict(base=1e4)
    dev = [cache.cuda(), kn.cuda(), vn.cuda()]
    qs = [q.cuda(), (q * 0.5).cuda()]
    x = [torch.randn(300, 40001, generator=torch.Generator().manual_seed(i)).cuda() for i in range(2)]
    toks = torch.arange(300, dtype=torch.int32).cuda()

    def run(i, ws, lp_ws, outs):
        a = (qs[i], dev[0], i32t, dev[1], dev[2], None, lt, cut, outs[0])
        pkg.kv4_verify(*a, ws, int(cu[-1]), B, rope, 0.1, order=ORDER["causal"])
        pkg.token_logprobs(x[i], toks, *outs[1:], lp_ws)

    i32t, lt, cut, rope = i32(table), i32(lens), i32(cu), pkg.rope_spec(**spec)

    def outputs():
        return (torch.empty_like(qs[0]), torch.empty(300, device="cuda"), torch.empty(300, dtype=torch.int32, device="cuda"),
                torch.empty(300, device="cuda"), torch.empty(300, 8, dtype=torch.int32, device="cuda"), torch.empty(300, 8, device="cuda"))

    o = [outputs() for _ in range(4)]
    size = pkg.kv4_verify_workspace_size(qs[0], dev[0], i32t, dev[1], dev[2], None, lt, cut, o[0][0], int(cu[-1]), B, rope, 0.1,
                                         order=ORDER["causal"])
    lp_size = pkg.token_logprobs_workspace_size(x[0], toks, *o[0][1:])
    ws = [(workspace(size), workspace(lp_size)) for _ in range(2)]
    for i in range(2):
        run(i, *ws[0], o[i])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                run(i, *ws[i], o[2 + i])
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(a, b) for a, b in zip(o[i], o[2 + i]))


@pytest.mark.parametrize("B,batch", [(1, 700), (4, 90), (16, 40)])
def test_more_units_than_fit_at_once(B, batch):
    """Several waves of CTAs, whole and cut units, ragged lengths, captured before any eager call of the shape."""
    g = torch.Generator().manual_seed(B)
    lens = torch.randint(0, 600, (batch,), generator=g).tolist()
    cache, table, cu, q, kn, vn, tau = case(B, lens, [B] * batch, "paired" if B > 1 else "causal", "bf16", 4, 2, 128)
    order, spec = "paired" if B > 1 else "causal", dict(base=1e4)
    args = [q.cuda(), cache.cuda(), i32(table), kn.cuda(), vn.cuda(), i32(tau), i32(lens), i32(cu)]
    out = torch.empty_like(args[0])
    rope = pkg.rope_spec(**spec)
    ws = workspace(pkg.kv4_verify_workspace_size(*args, out, B * batch, B, rope, 0.1, order=ORDER[order]))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pkg.kv4_verify(*args, out, ws, B * batch, B, rope, 0.1, order=ORDER[order])
    for _ in range(2):
        out.fill_(7)
        graph.replay()
    assert pkg.read_status(ws) == 0
    some = sorted(torch.randperm(batch, generator=g)[:12].tolist())
    per = 2 if order == "paired" else 1
    rows = torch.cat([torch.arange(per * B) + per * B * b for b in some])
    t = torch.stack([table[b] for b in some])
    want, off = ref.verify(q[rows], cache, t, kn[rows], vn[rows], torch.cat([tau[B * b:B * b + B] for b in some]), [lens[b] for b in some],
                           cu_of([B] * 12), spec, 0.1, order, 0, 2.0 ** -11)
    close(out[rows.cuda()], want, off, "bf16")


def test_other_devices_are_refused():
    """Tensors on the CPU beside ones on the GPU: an error, no launch."""
    cache, table, cu, q, kn, vn, tau = case(1, (20,), [2], "causal", "bf16", 4, 1, 64)
    rope, out, ws = pkg.rope_spec(), torch.empty_like(q).cuda(), workspace(1 << 20)
    good = [q.cuda(), cache.cuda(), i32(table), kn.cuda(), vn.cuda(), None, i32([20]), i32([0, 2]), out, ws]
    for i in (0, 1, 2, 3, 4, 6, 7, 8, 9):
        bad = list(good)
        bad[i] = bad[i].cpu()
        with pytest.raises(ValueError):
            pkg.kv4_verify(*bad, 2, 2, rope, 0.1, order=ORDER["causal"])
    x, t = torch.zeros(2, 9).cuda(), torch.zeros(2, dtype=torch.int32).cuda()
    for bad in ((x.cpu(), t, x[:, 0].contiguous()), (x, t.cpu(), x[:, 0].contiguous()), (x, t, torch.zeros(2))):
        with pytest.raises(ValueError):
            pkg.token_logprobs(*bad, None, None, None, None, ws)
    k = torch.zeros(3, 1, 64).cuda()
    for i in range(5):
        a = [cache.cuda(), i32(table), i32([0]), i32([0, 3]), k]
        a[i] = a[i].cpu()
        with pytest.raises(ValueError):
            pkg.kv4_read(*a, None, ws)
        with pytest.raises(ValueError):
            pkg.kv4_append(a[4], k, a[2], a[3], a[0], a[1], ws, rope)


@pytest.mark.parametrize("B", [3, 6, 16])
def test_many_calls_wait_for_nothing_in_vain(B):
    """Some thousand CTAs of ragged lengths: no call's waits run out, and each gives what the first gave."""
    g = torch.Generator().manual_seed(B)
    lens = torch.randint(0, 2500, (300,), generator=g).tolist()
    cache, table, cu, q, kn, vn, tau = case(B, lens, [B] * 300, "paired", "bf16", 4, 1, 128)
    args = [q.cuda(), cache.cuda(), i32(table), kn.cuda(), vn.cuda(), i32(tau), i32(lens), i32(cu)]
    outs = [torch.empty_like(args[0]) for _ in range(2)]
    rope = pkg.rope_spec()
    ws = workspace(pkg.kv4_verify_workspace_size(*args, outs[0], B * 300, B, rope, 0.1, order=ORDER["paired"]))
    for i in range(40):
        pkg.kv4_verify(*args, outs[min(i, 1)], ws, B * 300, B, rope, 0.1, order=ORDER["paired"], wait_polls=50000)
        if i:
            assert torch.equal(outs[0], outs[1])
    assert pkg.read_status(ws) == 0
