"""Dense attention over packed sequences, forward and backward, on the GPU
against the fp64 oracle and its derived tolerances (see dense_oracle), and a
whole serving and training run of the dense operators together.
L2 errors: each of the roundings on the way (P or dZ, and the result) has a
root mean square of at most 2^-8 / sqrt(3) = 2.3e-3 of the value: out and dv
stay below 3.2e-3 (4e-3 asked for).  dq and dk also carry D's error, which
does not shrink with dZ where dP and D nearly cancel: their bound adds the
oracle's share of it in the same norm."""
import numpy as np
import pytest
import torch

import block_sparse_long_08_b200.msa as M
import oracle.dense_oracle as O

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16 = torch.bfloat16


def f64(t):
    return t.detach().to("cpu", torch.float64).numpy()


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def packed(lens_q, lens_k, G, R, seed=0, tail=0, gain=1.0):
    """Packed inputs; `tail` rows of NaN behind the last sequence."""
    gen = torch.Generator().manual_seed(seed)
    cq, ck = [0] + np.cumsum(lens_q).tolist(), [0] + np.cumsum(lens_k).tolist()
    x = {"q": gain * torch.randn(cq[-1] + tail, G * R, 128, generator=gen),
         "k": torch.randn(ck[-1] + tail, G, 128, generator=gen),
         "v": torch.randn(ck[-1] + tail, G, 128, generator=gen),
         "dout": torch.randn(cq[-1] + tail, G * R, 128, generator=gen)}
    for n in x:
        x[n] = x[n].to(BF16)
        x[n][(cq if n in ("q", "dout") else ck)[-1]:] = float("nan")
    return {n: t.to(DEV) for n, t in x.items()}, cq, ck


def run(x, cq, ck, scale=0.0, ws=None):
    out = torch.full_like(x["q"], 7.0)
    lse = torch.full(x["q"].shape[:2], 7.0, device=DEV)
    M.msa_dense_attn_varlen(x["q"], x["k"], x["v"], i32(cq), i32(ck), out=out, lse=lse, scale=scale, ws=ws)
    return out, lse


def check_forward(x, cq, ck, out, lse, scale=None):
    nq, nk = cq[-1], ck[-1]
    ref, rl, tol, lt = O.dense(f64(x["q"])[:nq], f64(x["k"])[:nk], f64(x["v"])[:nk], cq, ck, scale)
    got, gl = f64(out), f64(lse)
    assert (got[nq:] == 7).all() and (gl[nq:] == 7).all(), "rows behind the last sequence changed"
    err = np.abs(got[:nq] - ref)
    assert (err <= tol).all(), (np.nanmax(err - tol), np.argwhere(~(err <= tol))[:4])
    assert np.linalg.norm(err) <= 4e-3 * np.linalg.norm(ref)
    gl = gl[:nq]
    assert np.array_equal(np.isneginf(gl), np.isneginf(rl))
    fin = np.isfinite(rl)
    le = np.abs(gl[fin] - rl[fin])
    assert (le <= lt[fin]).all(), (le - lt[fin]).max()


def check_backward(x, cq, ck, out, lse, scale=None, ws=None):
    nq, nk = cq[-1], ck[-1]
    g = {"dq": torch.full_like(x["q"], 7.0), "dk": torch.full_like(x["k"], 7.0), "dv": torch.full_like(x["v"], 7.0)}
    M.msa_dense_attn_varlen_backward(x["q"], x["k"], x["v"], out, lse, x["dout"], i32(cq), i32(ck), **g,
                                     scale=scale or 0.0, ws=ws)
    ref, tol = O.dense_backward(f64(x["q"])[:nq], f64(x["k"])[:nk], f64(x["v"])[:nk], f64(x["dout"])[:nq], cq, ck,
                                scale)
    for n, rows in (("dq", nq), ("dk", nk), ("dv", nk)):
        got = f64(g[n])
        assert (got[rows:] == 7).all(), n
        err = np.abs(got[:rows] - ref[n])
        assert (err <= tol[n]).all(), (n, np.nanmax(err - tol[n]), np.argwhere(~(err <= tol[n]))[:4])
        # D's share: |dout . out| carries out's roundings, 2^-8 / sqrt(3) each,
        # of 128 independent products; at most its worst case over sqrt(128)
        part = np.linalg.norm(tol[n]) / np.sqrt(128) if n != "dv" else 0.0
        assert np.linalg.norm(err) <= 4e-3 * np.linalg.norm(ref[n]) + part, n
    return g


CASES = [
    ([1], [1], 1, 1), ([1, 1, 1], [1, 5, 200], 2, 4), ([128], [128], 1, 1), ([129], [129], 1, 4),
    ([5, 0, 130, 377], [5, 0, 130, 377], 2, 4), ([64, 65, 63], [64, 65, 63], 1, 16), ([300], [300], 3, 2),
    ([100, 40], [700, 40], 2, 8), ([33, 257], [161, 513], 1, 4), ([0, 3], [9, 3], 1, 2),
    ([50, 20], [20, 50], 2, 4),      # more queries than keys: the first rows see none
    ([7, 9], [0, 0], 1, 4),          # no keys at all
    ([700], [1000], 1, 8), ([1100], [1100], 2, 1), ([1] * 150, [1] * 150, 1, 2),
]


@pytest.mark.parametrize("lens_q,lens_k,G,R", CASES)
def test_forward_and_backward(lens_q, lens_k, G, R):
    x, cq, ck = packed(lens_q, lens_k, G, R, seed=R, tail=5)
    ws = M.new_dense_workspace(M.MSA_OP_DENSE_VARLEN, x["q"], x["k"], len(lens_q))
    out, lse = run(x, cq, ck, ws=ws)
    assert M.msa_read_status(ws) == M.MSA_OK
    check_forward(x, cq, ck, out, lse)
    wsb = M.new_dense_workspace(M.MSA_OP_DENSE_VARLEN_BACKWARD, x["q"], x["k"], len(lens_q))
    check_backward(x, cq, ck, out, lse, ws=wsb)
    assert M.msa_read_status(wsb) == M.MSA_OK


@pytest.mark.parametrize("gain,scale", [(30.0, None), (1.0, 1.0), (0.0, None)])
def test_peaked_and_flat_rows(gain, scale):
    """Scores far apart (the maximum moves), a scale of one, and all equal."""
    x, cq, ck = packed([400, 90], [500, 90], 1, 4, seed=2, gain=gain)
    out, lse = run(x, cq, ck, scale=scale or 0.0)
    check_forward(x, cq, ck, out, lse, scale)
    check_backward(x, cq, ck, out, lse, scale)


def test_rising_scores_rescale_every_tile():
    n = 1500
    x, cq, ck = packed([n], [n], 1, 2, seed=4)
    x["k"].zero_()
    x["k"][:, 0, 0] = (torch.arange(n, device=DEV) / 50).to(BF16)
    x["q"].zero_()
    x["q"][:, 0, 0], x["q"][:, 1, 0] = 20.0, -20.0
    out, lse = run(x, cq, ck)
    check_forward(x, cq, ck, out, lse)


def test_other_sequences_do_not_leak():
    """A neighbour full of NaN and infinities changes nothing."""
    lens = [100, 61, 200]
    x, cq, ck = packed(lens, lens, 2, 4, seed=5)
    out, lse = run(x, cq, ck)
    g = check_backward(x, cq, ck, out, lse)
    for bad in (float("nan"), float("inf"), -float("inf")):
        y = {n: t.clone() for n, t in x.items()}
        for n in y:
            y[n][100:161] = bad
        o2, l2 = run(y, cq, ck)
        h = {"dq": torch.empty_like(y["q"]), "dk": torch.empty_like(y["k"]), "dv": torch.empty_like(y["v"])}
        M.msa_dense_attn_varlen_backward(y["q"], y["k"], y["v"], o2, l2, y["dout"], i32(cq), i32(ck), **h)
        for a, b in [(out, o2), (lse, l2)] + [(g[n], h[n]) for n in g]:
            assert torch.equal(a[:100], b[:100]) and torch.equal(a[161:], b[161:])


def test_bad_starts_are_refused_whole():
    x, _, _ = packed([50, 50], [50, 50], 1, 2)
    for cq, ck in [([0, 60, 50], [0, 50, 100]), ([0, 50, 101], [0, 50, 100]), ([-1, 50, 100], [0, 50, 100]),
                   ([0, 50, 100], [0, 50, 101])]:
        ws = M.new_dense_workspace(M.MSA_OP_DENSE_VARLEN_BACKWARD, x["q"], x["k"], 2)
        out, lse = run(x, cq, ck, ws=ws)
        assert M.msa_read_status(ws) == M.MSA_ERR_DEVICE_INPUT
        assert (out == 7).all() and (lse == 7).all()
        g = {"dq": torch.full_like(x["q"], 7.0), "dk": torch.full_like(x["k"], 7.0), "dv": torch.full_like(x["v"], 7.0)}
        M.msa_dense_attn_varlen_backward(x["q"], x["k"], x["v"], out, lse, x["dout"], i32(cq), i32(ck), **g, ws=ws)
        assert M.msa_read_status(ws) == M.MSA_ERR_DEVICE_INPUT
        assert all((t == 7).all() for t in g.values())


def test_repeats_bit_for_bit_and_starts_behind_zero():
    lens = [900, 300, 1200]
    x, cq, ck = packed(lens, lens, 2, 4, seed=6)
    a = run(x, cq, ck)
    ga = M.msa_dense_attn_varlen_backward(x["q"], x["k"], x["v"], *a, x["dout"], i32(cq), i32(ck))
    for _ in range(3):
        b = run(x, cq, ck)
        gb = M.msa_dense_attn_varlen_backward(x["q"], x["k"], x["v"], *b, x["dout"], i32(cq), i32(ck))
        assert all(torch.equal(s, t) for s, t in zip(a + tuple(ga), b + tuple(gb)))
    # the first start need not be 0: rows before it are left alone
    b = run(x, cq[1:], ck[1:])
    assert (b[0][:900] == 7).all() and torch.equal(b[0][900:], a[0][900:])


def test_long_sequence_sampled():
    """8K tokens: sampled rows of the forward and dq, sampled keys of dk, dv."""
    n, G, R = 8192, 2, 4
    x, cq, ck = packed([n], [n], G, R, seed=7)
    out, lse = run(x, cq, ck)
    dq, dk, dv = M.msa_dense_attn_varlen_backward(x["q"], x["k"], x["v"], out, lse, x["dout"], i32(cq), i32(ck))
    w = {m: t.double() for m, t in x.items()}
    for h in (0, 5):
        k, v = w["k"][:, h // R], w["v"][:, h // R]
        z = (w["q"][:, h] @ k.t()) / 128 ** 0.5
        z.masked_fill_(torch.ones_like(z, dtype=torch.bool).triu(1), -float("inf"))
        p = torch.softmax(z, -1)
        o = p @ v
        assert (out[:, h].double() - o).norm() <= 4e-3 * o.norm()
        assert (lse[:, h].double() - torch.logsumexp(z, -1)).abs().max() < 1e-4
        dp = w["dout"][:, h] @ v.t()
        ds = p * (dp - (w["dout"][:, h] * o).sum(-1, keepdim=True))
        r = ds @ k / 128 ** 0.5
        assert (dq[:, h].double() - r).norm() <= 6e-3 * r.norm()
    rk, rv = torch.zeros_like(w["k"][:, 0]), torch.zeros_like(w["k"][:, 0])
    for h in range(R):
        k, v = w["k"][:, 0], w["v"][:, 0]
        z = ((w["q"][:, h] @ k.t()) / 128 ** 0.5).masked_fill_(torch.ones(n, n, dtype=torch.bool, device=DEV).triu(1), -float("inf"))
        p = torch.softmax(z, -1)
        dp = w["dout"][:, h] @ v.t()
        ds = p * (dp - (p * dp).sum(-1, keepdim=True))
        rk += ds.t() @ w["q"][:, h] / 128 ** 0.5
        rv += p.t() @ w["dout"][:, h]
    assert (dk[:, 0].double() - rk).norm() <= 6e-3 * rk.norm()
    assert (dv[:, 0].double() - rv).norm() <= 6e-3 * rv.norm()


def test_captured_and_replayed_with_other_lengths():
    """One captured graph serves other lengths, positions and pages."""
    lens = [60, 200, 40]
    x, cq, ck = packed(lens, lens, 1, 4, seed=8)
    dcq, dck = i32(cq), i32(ck)
    out, lse = torch.zeros_like(x["q"]), torch.zeros(x["q"].shape[:2], device=DEV)
    wf = M.new_dense_workspace(M.MSA_OP_DENSE_VARLEN, x["q"], x["k"], 3)
    wb = M.new_dense_workspace(M.MSA_OP_DENSE_VARLEN_BACKWARD, x["q"], x["k"], 3)
    g = {"dq": torch.zeros_like(x["q"]), "dk": torch.zeros_like(x["k"]), "dv": torch.zeros_like(x["v"])}

    def step():
        M.msa_dense_attn_varlen(x["q"], x["k"], x["v"], dcq, dck, out=out, lse=lse, ws=wf)
        M.msa_dense_attn_varlen_backward(x["q"], x["k"], x["v"], out, lse, x["dout"], dcq, dck, ws=wb, **g)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        step()
        s.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            step()
    for lens in ([60, 200, 40], [1, 150, 149], [300, 0, 0]):
        c = [0] + np.cumsum(lens).tolist()
        dcq.copy_(i32(c))
        dck.copy_(i32(c))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        want = run(x, c, c)
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
        check_forward(x, c, c, out, lse)
        wg = M.msa_dense_attn_varlen_backward(x["q"], x["k"], x["v"], out, lse, x["dout"], i32(c), i32(c))
        assert all(torch.equal(a, b) for a, b in zip(g.values(), wg))


@pytest.mark.parametrize("fp8", [False, True])
def test_prompt_then_steps_equal_the_whole_sequence(fp8):
    """Prompts appended and attended to, then tokens one by one: as a serving
    loop runs it, on a stream of its own, against dense attention in 64 bits
    over the whole rotated sequences."""
    G, R, page, steps = 2, 4, 16, 4
    prompts = [37, 5, 130]
    total = [n + steps for n in prompts]
    gen = torch.Generator().manual_seed(12)
    f = (10000.0 ** (-torch.arange(64).float() / 64)).to(DEV)
    full = {n: [torch.randn(t, h, 128, generator=gen).to(BF16) for t in total]
            for n, h in (("q", G * R), ("k", G), ("v", G))}
    rot = {n: [O.rotate(f64(t), np.arange(t.shape[0]), f64(f), 128, False) for t in full[n]] for n in ("q", "k")}
    need = [-(-t // page) for t in total]
    num = sum(need)
    ids = torch.randperm(num, generator=gen).to(torch.int32)
    table = torch.full((3, max(need)), -1, dtype=torch.int32)
    for b, at in enumerate(np.cumsum([0] + need[:-1])):
        table[b, :need[b]] = ids[at:at + need[b]]
    table = table.to(DEV)
    kind = torch.uint8 if fp8 else BF16
    kp, vp = (torch.full((num, page, G, 128), 0x7F if fp8 else float("nan"), dtype=kind, device=DEV) for _ in range(2))
    ks, vs = (torch.full((num, page, G), float("nan"), device=DEV) if fp8 else None for _ in range(2))
    sc = {"k_scale": ks, "v_scale": vs}
    s = torch.cuda.Stream()
    got = [[] for _ in range(3)]
    with torch.cuda.stream(s):
        pk = {n: torch.cat([t[:p] for t, p in zip(full[n], prompts)]).to(DEV) for n in full}
        cu = i32([0] + np.cumsum(prompts).tolist())
        k_rot = torch.empty_like(pk["k"])
        q_rot = M.msa_paged_append(pk["k"], pk["v"], kp, vp, table, i32(prompts), cu_new=cu, q=pk["q"], k_out=k_rot,
                                   inv_freq=f, **sc)
        out = M.msa_dense_attn_varlen(q_rot, k_rot, pk["v"], cu, cu)
        for b in range(3):
            got[b].append(out[cu[b]:cu[b + 1]])
        lens = i32(prompts)
        for i in range(steps):
            lens += 1
            now = {n: torch.stack([t[p + i] for t, p in zip(full[n], prompts)]).to(DEV) for n in full}
            M.msa_paged_append(now["k"], now["v"], kp, vp, table, lens, q=now["q"], q_out=now["q"], inv_freq=f, **sc)
            o = M.msa_paged_attn_decode(now["q"], kp, vp, table, lens, **sc)
            for b in range(3):
                got[b].append(o[b:b + 1])
    s.synchronize()
    for b in range(3):
        ref = O.dense(rot["q"][b], rot["k"][b], f64(full["v"][b]), [0, total[b]], [0, total[b]])[0]
        err = f64(torch.cat(got[b])) - ref
        # q, k and v are rounded too: five roundings of 2.3e-3 rms give 5e-3 on
        # scores of order one; 8-bit steps (2^-4 / sqrt(3) = 3.6e-2) on the decode rows
        p = prompts[b]
        assert np.linalg.norm(err[:p]) <= 1.2e-2 * np.linalg.norm(ref[:p])
        assert np.linalg.norm(err[p:]) <= (0.12 if fp8 else 1.2e-2) * np.linalg.norm(ref[p:])


def test_rows_behind_two_billion_values():
    """Packed rows whose element offsets pass 2^31: sequences at the end give
    what they give alone."""
    H, G, n, B = 64, 4, 128, 2080
    gen = torch.Generator(device=DEV).manual_seed(3)
    lens = [n] * (B - 1) + [77]
    cu = [0] + np.cumsum(lens).tolist()
    q, dout = (torch.randn(cu[-1], H, 128, device=DEV, dtype=BF16, generator=gen) for _ in range(2))
    k, v = (torch.randn(cu[-1], G, 128, device=DEV, dtype=BF16, generator=gen) for _ in range(2))
    assert q.numel() > 2 ** 31
    out, lse = M.msa_dense_attn_varlen(q, k, v, i32(cu), i32(cu), want_lse=True)
    g = M.msa_dense_attn_varlen_backward(q, k, v, out, lse, dout, i32(cu), i32(cu))
    for b in (0, 1000, B - 2, B - 1):
        s = slice(cu[b], cu[b + 1])
        c = [0, lens[b]]
        o, ls = M.msa_dense_attn_varlen(q[s], k[s], v[s], i32(c), i32(c), want_lse=True)
        assert torch.equal(o, out[s]) and torch.equal(ls, lse[s]), b
        h = M.msa_dense_attn_varlen_backward(q[s], k[s], v[s], o, ls, dout[s], i32(c), i32(c))
        assert all(torch.equal(x, y[s]) for x, y in zip(h, g)), b


def test_many_sequences_and_more_than_the_plan_holds_at_once():
    """3000 sequences of 0 to 5 tokens: the plan walks them in chunks."""
    rng = np.random.default_rng(4)
    lens = rng.integers(0, 6, 3000).tolist()
    x, cq, ck = packed(lens, lens, 1, 4, seed=9, tail=3)
    out, lse = run(x, cq, ck)
    check_forward(x, cq, ck, out, lse)
    check_backward(x, cq, ck, out, lse)


def test_forward_without_lse_and_on_a_given_stream():
    lens = [200, 90]
    x, cq, ck = packed(lens, lens, 2, 4, seed=10)
    want, _ = run(x, cq, ck)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    out = M.msa_dense_attn_varlen(x["q"], x["k"], x["v"], i32(cq), i32(ck), stream=s)
    s.synchronize()
    assert torch.equal(out, want)


@pytest.mark.parametrize("n,G,R", [(128, 4, 16), (40, 2, 4), (200, 8, 8), (300, 4, 1)])
def test_short_sequences_back_to_back_repeat(n, G, R):
    """Many short items per CTA, one after the other through every hand-over
    between the warps: 30 runs give the same bits."""
    lens = [n + i % 3 for i in range(150)]
    x, cq, ck = packed(lens, lens, G, R, seed=12)
    a = run(x, cq, ck)
    ga = M.msa_dense_attn_varlen_backward(x["q"], x["k"], x["v"], *a, x["dout"], i32(cq), i32(ck))
    one = slice(0, lens[0])
    o = M.msa_dense_attn_varlen(x["q"][one], x["k"][one], x["v"][one], i32([0, lens[0]]), i32([0, lens[0]]))
    assert torch.equal(o, a[0][one])
    for _ in range(30):
        b = run(x, cq, ck)
        gb = M.msa_dense_attn_varlen_backward(x["q"], x["k"], x["v"], *b, x["dout"], i32(cq), i32(ck))
        assert all(torch.equal(s, t) for s, t in zip(a + tuple(ga), b + tuple(gb)))


def test_bad_starts_of_a_large_batch_are_refused_whole():
    """The listed plan's refusal in the forward (more sequences than a call
    plans for itself)."""
    lens = [20] * 50
    x, cq, ck = packed(lens, lens, 1, 2)
    cq[30] = cq[29] - 1
    ws = M.new_dense_workspace(M.MSA_OP_DENSE_VARLEN, x["q"], x["k"], 50)
    out, lse = run(x, cq, ck, ws=ws)
    assert M.msa_read_status(ws) == M.MSA_ERR_DEVICE_INPUT
    assert (out == 7).all() and (lse == 7).all()


@pytest.mark.parametrize("R", [1, 4, 16])
def test_nan_in_a_query_stays_in_its_row(R):
    lens = [3, 300, 40]
    x, cq, ck = packed(lens, lens, 2, R, seed=R)
    out, lse = run(x, cq, ck)
    hit = torch.zeros_like(lse, dtype=torch.bool)
    for i, h in ((1, 0), (150, 2 * R - 1), (302, R)):
        x["q"][i, h, 7] = float("nan")
        hit[i, h] = True
    o, ls = run(x, cq, ck)
    assert torch.isnan(o[hit]).all() and torch.isnan(ls[hit]).all()
    assert torch.equal(o[~hit], out[~hit]) and torch.equal(ls[~hit], lse[~hit])


def test_what_a_call_allocates_belongs_to_the_given_stream():
    """The stream is busy while the call is made, and other work of the current
    one takes memory of the same sizes at once."""
    lens = [600, 90, 1]
    x, cq, ck = packed(lens, lens, 2, 4, seed=12)
    out, lse = run(x, cq, ck)
    grads = M.msa_dense_attn_varlen_backward(x["q"], x["k"], x["v"], out, lse, x["dout"], i32(cq), i32(ck))
    nk = x["k"].shape[0]
    table = torch.arange(64, dtype=torch.int32, device=DEV).reshape(1, 64)
    kp, vp = (torch.zeros(64, 16, 2, 128, dtype=BF16, device=DEV) for _ in range(2))
    n = i32([nk])
    M.msa_paged_append(x["k"], x["v"], kp, vp, table, n, cu_new=i32([0, nk]))
    one = M.msa_paged_attn_decode(x["q"][:1], kp, vp, table, n)
    cqd, ckd = i32(cq), i32(ck)
    s = torch.cuda.Stream()

    def calls():
        o, ls = M.msa_dense_attn_varlen(x["q"], x["k"], x["v"], cqd, ckd, want_lse=True, stream=s)
        g = M.msa_dense_attn_varlen_backward(x["q"], x["k"], x["v"], out, lse, x["dout"], cqd, ckd, stream=s)
        return (o, ls) + tuple(g) + (M.msa_paged_attn_decode(x["q"][:1], kp, vp, table, n, stream=s),)

    calls()                                   # (freed memory of these sizes is there to be taken)
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(20_000_000)
    got = calls()
    junk = [torch.full((2 ** i,), 255, dtype=torch.uint8, device=DEV) for i in range(8, 22) for _ in range(4)]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, (out, lse) + tuple(grads) + (one,)))
    assert all((j == 255).all() for j in junk)


def test_a_refused_batch_without_a_workspace_gives_zeros():
    """Results that the call allocates hold nothing of older memory."""
    x, _, _ = packed([50, 50], [50, 50], 1, 2)
    cq, ck = i32([0, 60, 50]), i32([0, 50, 100])
    for _ in range(3):
        junk = [torch.full_like(x[n], 7.0) for n in ("q", "q", "k", "k", "k")] + [torch.full((100, 2), 7.0, device=DEV)]
        del junk
        out, lse = M.msa_dense_attn_varlen(x["q"], x["k"], x["v"], cq, ck, want_lse=True)
        assert (out == 0).all() and (lse == 0).all()
        del out, lse
        out, lse = torch.zeros_like(x["q"]), torch.zeros(100, 2, device=DEV)
        junk = [torch.full_like(x[n], 7.0) for n in ("q", "q", "k", "k", "k")]
        del junk
        grads = M.msa_dense_attn_varlen_backward(x["q"], x["k"], x["v"], out, lse, x["dout"], cq, ck)
        assert all((t == 0).all() for t in grads)
        del grads


@pytest.mark.parametrize("R", [1, 4, 16])
@pytest.mark.parametrize("lens_q,lens_k", [([7, 9], [0, 0]), ([0, 0], [7, 9]), ([300], [0]), ([0], [300]),
                                           ([1] * 40, [0] * 40), ([0] * 40, [200] * 40)])
def test_no_keys_or_no_queries(lens_q, lens_k, R):
    """Buffers of no rows at all: results are zero (lse -inf), and written."""
    x, cq, ck = packed(lens_q, lens_k, 2, R, seed=R, tail=0)
    ws = M.new_dense_workspace(M.MSA_OP_DENSE_VARLEN, x["q"], x["k"], len(lens_q))
    out, lse = run(x, cq, ck, ws=ws)
    assert (out == 0).all() and torch.isneginf(lse).all()
    wsb = M.new_dense_workspace(M.MSA_OP_DENSE_VARLEN_BACKWARD, x["q"], x["k"], len(lens_q))
    g = {n: torch.full_like(x[n[1:]], 7.0) for n in ("dq", "dk", "dv")}
    M.msa_dense_attn_varlen_backward(x["q"], x["k"], x["v"], out, lse, x["dout"], i32(cq), i32(ck), ws=wsb, **g)
    assert all((t == 0).all() for t in g.values())
    assert M.msa_read_status(ws) == M.MSA_OK and M.msa_read_status(wsb) == M.MSA_OK
