"""Paged cache append and single-token attention on the GPU against the fp64
oracle, whose tolerances are derived from the roundings (see dense_oracle).
Append: one rounding to bf16 (or E4M3) of a value that is off by at most
2^-20 of its pair's length (fp32 rotation by a cosine and sine good to 2^-22,
two products and a sum).  L2 errors: independent roundings of at most 2^-8
each have a root mean square of at most 2^-8 / sqrt(3) = 2.3e-3, so two of
them (weights and output) stay below 3.2e-3; 4e-3 is asked for."""
import numpy as np
import pytest
import torch

import block_sparse_long_08_b200.msa as M
import oracle.dense_oracle as O
from oracle.msa_oracle import e4m3_to_f64

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16 = torch.bfloat16


def f64(t):
    return t.detach().to("cpu", torch.float64).numpy()


def make_cache(lens, G, page, fp8, seed=0, extra=2, cols=None, junk=True):
    """Scattered pages; every row of the pool that no token owns is NaN."""
    gen = torch.Generator().manual_seed(seed)
    need = [-(-max(n, 0) // page) for n in lens]
    num = sum(need) + extra
    ids = torch.randperm(num, generator=gen).to(torch.int32)
    cols = cols or max(need + [1]) + 1
    table = torch.full((len(lens), cols), -7, dtype=torch.int32)
    own = torch.zeros(num, page, dtype=torch.bool)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = ids[at:at + n]
        for t in range(max(lens[b], 0)):
            own[table[b, t // page], t % page] = True
        at += n
    c = {"table": table.to(DEV), "own": own}
    for x in "kv":
        w = torch.randn(num, page, G, 128, generator=gen)
        if fp8:
            codes, scale = w.to(torch.float8_e4m3fn).view(torch.uint8), torch.rand(num, page, G, generator=gen) + 0.5
            if junk:
                codes[~own], scale[~own] = 0x7F, float("nan")
            c[x], c[x + "s"] = codes.to(DEV), scale.to(DEV)
        else:
            w = w.to(BF16)
            if junk:
                w[~own] = float("nan")
            c[x], c[x + "s"] = w.to(DEV), None
    return c


def cache_f64(c, x):
    if c[x + "s"] is None:
        return f64(c[x])
    return e4m3_to_f64(c[x].cpu().numpy()) * f64(c[x + "s"])[..., None]


def gathered(c, x, b, n):
    page = c[x].shape[1]
    t = torch.arange(n, device=DEV)
    at = (c["table"][b, t // page].long(), t % page)
    return cache_f64({x: c[x][at], x + "s": None if c[x + "s"] is None else c[x + "s"][at]}, x)


def decode(c, q, lens, **kw):
    t = torch.tensor(lens, dtype=torch.int32, device=DEV)
    return M.msa_paged_attn_decode(q, c["k"], c["v"], c["table"], t, k_scale=c["ks"], v_scale=c["vs"],
                                   want_lse=True, **kw)


def check_decode(c, q, lens, out, lse, scale=None, skip=None):
    G = c["k"].shape[2]
    B, H, d = q.shape
    ref, tol = np.zeros(q.shape), np.zeros(q.shape)
    for b, n in enumerate(lens):
        k, v = gathered(c, "k", b, n), gathered(c, "v", b, n)
        if skip is not None:
            k, v = k[skip[b]], v[skip[b]]
            n = k.shape[0]
        o, ls, t, lt = O.dense(f64(q[b])[None], k, v, [0, 1], [0, n], scale)
        ref[b], tol[b] = o[0], t[0]
        got = f64(lse[b])
        assert np.array_equal(np.isinf(got), np.isinf(ls[0])), b
        fin = np.isfinite(got)
        assert (np.abs(got[fin] - ls[0][fin]) <= lt[0][fin]).all(), (b, np.abs(got[fin] - ls[0][fin]).max())
    err = np.abs(f64(out) - ref)
    assert (err <= tol).all(), (err - tol).max()
    assert np.linalg.norm(err) <= 4e-3 * np.linalg.norm(ref)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("G,R,page", [(2, 4, 64), (1, 16, 16), (8, 1, 32), (3, 2, 128), (2, 8, 256)])
def test_decode_matches_oracle(G, R, page, fp8):
    lens = [1, 0, 15, 16, 17, 63, 64, 65, 300, 1023]
    c = make_cache(lens, G, page, fp8, seed=G * R)
    q = torch.randn(len(lens), G * R, 128, generator=torch.Generator().manual_seed(1)).to(BF16).to(DEV)
    out, lse = decode(c, q, lens)
    check_decode(c, q, lens, out, lse)
    assert (f64(out)[1] == 0).all() and np.isneginf(f64(lse)[1]).all()


@pytest.mark.parametrize("lens,G,R", [([40000], 1, 4), ([20000, 3, 9000], 2, 8), ([1], 1, 1),
                                      ([7] * 300, 1, 2), ([5000] * 5, 4, 16), ([2049] * 40, 8, 4)])
@pytest.mark.parametrize("fp8", [False, True])
def test_decode_long_and_many(lens, G, R, fp8):
    c = make_cache(lens, G, 32, fp8, seed=3)
    q = torch.randn(len(lens), G * R, 128, generator=torch.Generator().manual_seed(2)).to(BF16).to(DEV)
    ws = M.new_paged_workspace(M.MSA_OP_PAGED_DECODE, c["table"], 32, G * R, G)
    out, lse = decode(c, q, lens, ws=ws)
    check_decode(c, q, lens, out, lse)
    again, lse2 = decode(c, q, lens, ws=ws)
    assert torch.equal(out, again) and torch.equal(lse, lse2)
    assert M.msa_read_status(ws) == M.MSA_OK


def test_decode_large_scores_and_scale():
    """Scores of +-1000s: the running maximum carries them."""
    lens = [700, 64]
    c = make_cache(lens, 2, 64, False, seed=5, junk=True)
    q = (100 * torch.randn(2, 8, 128, generator=torch.Generator().manual_seed(2))).to(BF16).to(DEV)
    out, lse = decode(c, q, lens, scale=0.3)
    assert torch.isfinite(out).all()
    ref = np.zeros(q.shape)
    for b, n in enumerate(lens):
        ref[b] = O.dense(f64(q[b])[None], gathered(c, "k", b, n), gathered(c, "v", b, n), [0, 1], [0, n], 0.3)[0][0]
    # weights near 0 and 1: the score error itself is large here
    assert np.abs(f64(out) - ref).max() < 0.1


def test_decode_ascending_scores_move_the_maximum():
    """Every tile raises the maximum: rescaling happens all the way."""
    n = 3000
    c = make_cache([n], 1, 64, False, seed=6)
    k = torch.zeros_like(c["k"]).float()
    t = torch.arange(n, device=DEV)
    k[c["table"][0, t // 64].long(), t % 64, 0, 0] = torch.arange(n, device=DEV).float() / 100
    c["k"] = k.to(BF16)
    q = torch.zeros(1, 4, 128, device=DEV, dtype=BF16)
    q[..., 0] = torch.tensor([16.0, -16.0, 1.0, 0.0], device=DEV)
    out, lse = decode(c, q, [n])
    check_decode(c, q, [n], out, lse)


def test_decode_bad_lengths_and_pages():
    lens = [100, 200, 150]
    c = make_cache(lens, 2, 64, False, seed=7, junk=False)
    c["table"][1, 1] = c["k"].shape[0]          # tokens 64..127 of sequence 1 have no page
    q = torch.randn(3, 8, 128, generator=torch.Generator().manual_seed(2)).to(BF16).to(DEV)
    ws = M.new_paged_workspace(M.MSA_OP_PAGED_DECODE, c["table"], 64, 8, 2)
    out, lse = decode(c, q, [100, 200, 100000], ws=ws)
    assert M.msa_read_status(ws) == M.MSA_ERR_DEVICE_INPUT
    assert M.msa_read_status(ws) == M.MSA_OK
    assert (out[2] == 0).all() and torch.isneginf(lse[2]).all()
    c["table"][1, 1] = 0
    keep = [np.arange(100), np.r_[0:64, 128:200]]
    check_decode(c, q[:2], lens[:2], out[:2], lse[:2], skip=keep)
    out, lse = decode(c, q, [-1, 0, 150], ws=ws)
    assert M.msa_read_status(ws) == M.MSA_ERR_DEVICE_INPUT
    assert (out[:2] == 0).all() and torch.isfinite(lse[2]).all()


# ------------------------------------------------------------------- append

def check_append(lens, new, G, R, page, fp8, rot, inter, with_q=True, pad_rows=0, base=10000.0, inplace=False):
    gen = torch.Generator().manual_seed(11)
    one = new is None
    cu = None if one else [0] + list(np.cumsum(new))
    N = (len(lens) if one else cu[-1]) + pad_rows
    c = make_cache(lens, G, page, fp8, seed=8, junk=False)
    k, v = (torch.randn(N, G, 128, generator=gen).to(BF16).to(DEV) for _ in range(2))
    v[0, 0] = 0                                  # an all-zero row: scale 1
    q = torch.randn(N, G * R, 128, generator=gen).to(BF16).to(DEV) if with_q else None
    f = (base ** (-torch.arange(max(1, rot // 2)).float() / max(1, rot // 2))).to(DEV)
    before = {x: c[x].clone() for x in "kv"} | {x + "s": c[x + "s"].clone() if fp8 else None for x in "kv"}
    k0, q0 = k.clone(), q.clone() if with_q else None
    q_out = q if inplace else (torch.full_like(q, 3.0) if with_q else None)
    k_out = k if inplace else torch.full_like(k, 3.0)
    ws = M.new_paged_workspace(M.MSA_OP_PAGED_APPEND, c["table"], page, G * R, G)
    r = M.msa_paged_append(k, v, c["k"], c["v"], c["table"], torch.tensor(lens, dtype=torch.int32, device=DEV),
                           cu_new=None if one else torch.tensor(cu, dtype=torch.int32, device=DEV), q=q, q_out=q_out,
                           k_out=k_out, inv_freq=f if rot else None, rot_dim=rot, interleaved=inter,
                           k_scale=c["ks"], v_scale=c["vs"], ws=ws)
    assert M.msa_read_status(ws) == M.MSA_OK
    assert (r is None) == (not with_q)
    rows = O.token_rows(lens, cu)
    at, seq, pos = (np.array([x[i] for x in rows], dtype=int) for i in range(3))
    table = c["table"].cpu().numpy()
    pg, sl = table[seq, pos // page], pos % page
    if rows:
        assert np.array_equal(np.sort(pg * page + sl), np.unique(pg * page + sl))
    for x, src in (("k", k0), ("v", v)):
        want = f64(src)[at]
        size = np.abs(want)
        if x == "k":
            want = O.rotate(want, pos, f64(f), rot, inter)
            size = np.abs(want) + 0
            if rot:
                half = rot // 2
                i0 = np.arange(half) * (2 if inter else 1)
                i1 = i0 + (1 if inter else half)
                ln = np.hypot(want[..., i0], want[..., i1])
                size[..., i0], size[..., i1] = ln, ln
            out = f64(k_out)
            assert (np.abs(out[at] - want) <= O.U * np.abs(want) + 2.0 ** -20 * size).all()
            rest = np.setdiff1d(np.arange(N), at)
            assert np.array_equal(out[rest], (f64(k0) if inplace else np.full(out.shape, 3.0))[rest])
        got = cache_f64(c, x)[pg, sl]
        if fp8:
            amax = np.abs(want).max(-1)
            scale = np.where(amax > 0, amax / 448, 1.0)
            assert (np.abs(f64(c[x + "s"])[pg, sl] - scale) <= 2.0 ** -19 * scale).all()
            # half a step of a normal code is 2^-4 of it, of a subnormal one 2^-10 scales
            tol = np.maximum(2.0 ** -4 * np.abs(want), 2.0 ** -10 * scale[..., None]) * (1 + 2.0 ** -6)
            tol += 2.0 ** -18 * size
        else:
            tol = O.U * np.abs(want) + 2.0 ** -20 * size
        assert (np.abs(got - want) <= tol).all(), x
        touched = torch.zeros(c[x].shape[:2], dtype=torch.bool)
        touched[pg, sl] = True
        same = (c[x].cpu().view(torch.uint8) == before[x].cpu().view(torch.uint8)).flatten(2).all(-1)
        assert same[~touched].all(), "a row that no new token owns changed"
        if fp8:
            assert torch.equal(c[x + "s"].cpu()[~touched], before[x + "s"].cpu()[~touched])
    if with_q:
        want = O.rotate(f64(q0)[at], pos, f64(f), rot, inter)
        got = f64(r)
        assert (np.abs(got[at] - want) <= O.U * np.abs(want) + 2.0 ** -19 * np.abs(f64(q0)[at]).max()).all()
        rest = np.setdiff1d(np.arange(N), at)
        assert np.array_equal(got[rest], (f64(q0) if inplace else np.full(got.shape, 3.0))[rest])


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("rot,inter", [(128, False), (128, True), (64, False), (32, True), (16, False), (96, True),
                                       (112, False), (0, False)])
def test_append_rotations(rot, inter, fp8):
    check_append([70, 300, 33], [70, 5, 1], 2, 4, 64, fp8, rot, inter)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("G,R,page", [(1, 1, 16), (8, 4, 256), (3, 16, 32), (5, 2, 128)])
def test_append_steps_and_heads(G, R, page, fp8):
    check_append([1, 0, 16, 17, 512, 0, 1000], None, G, R, page, fp8, 128, False)


def test_append_padding_and_no_queries():
    check_append([20, 0, 9], [20, 4, 0], 2, 4, 16, False, 64, True, with_q=False, pad_rows=5)
    check_append([20, 0, 9], [20, 4, 9], 2, 4, 16, True, 64, False, pad_rows=3)
    check_append([40, 700], [40, 600], 2, 2, 64, False, 128, False, inplace=True)
    check_append([40, 700], [40, 600], 2, 2, 64, True, 128, True, inplace=True)


def test_append_many_rows():
    check_append([3000, 1501, 900], [2990, 1501, 3], 4, 2, 64, False, 128, False)


def test_append_far_positions():
    """Angles at a million tokens: fp32 products would be off by 0.06 rad."""
    n = 1 << 20
    page, G = 256, 1
    c = {x: torch.zeros(2, page, G, 128, dtype=BF16, device=DEV) for x in "kv"}
    table = torch.full((1, n // page), -1, dtype=torch.int32)
    table[0, -1] = 1
    f = (1e6 ** (-torch.arange(64).float() / 64)).to(DEV)
    k = torch.randn(3, G, 128, generator=torch.Generator().manual_seed(0)).to(BF16).to(DEV)
    M.msa_paged_append(k, k, c["k"], c["v"], table.to(DEV), torch.tensor([n], dtype=torch.int32, device=DEV),
                       cu_new=torch.tensor([0, 3], dtype=torch.int32, device=DEV), inv_freq=f)
    want = O.rotate(f64(k), np.arange(n - 3, n), f64(f), 128, False)
    got = f64(c["k"])[1, page - 3:]
    assert (np.abs(got - want) <= O.U * np.abs(want) + 2.0 ** -19 * np.abs(f64(k)).max()).all()


def test_append_bad_input_is_skipped():
    G, page = 1, 16
    k = torch.ones(6, G, 128, dtype=BF16, device=DEV)
    ws = torch.zeros(256, dtype=torch.uint8, device=DEV)

    def call(lens, cu, table):
        pages = torch.zeros(4, page, G, 128, dtype=BF16, device=DEV)
        t = torch.tensor(table, dtype=torch.int32, device=DEV)
        M.msa_paged_append(k, k, pages, pages.clone(), t, torch.tensor(lens, dtype=torch.int32, device=DEV),
                           cu_new=torch.tensor(cu, dtype=torch.int32, device=DEV), ws=ws)
        return M.msa_read_status(ws), (pages != 0).flatten(2).any(-1).nonzero().tolist()
    good = [[0], [1]]
    assert call([3, 3], [0, 3, 6], good) == (M.MSA_OK, [[0, 0], [0, 1], [0, 2], [1, 0], [1, 1], [1, 2]])
    bad = M.MSA_ERR_DEVICE_INPUT
    assert call([2, 3], [0, 3, 6], good) == (bad, [[1, 0], [1, 1], [1, 2]])    # fewer tokens than rows
    assert call([17, 3], [0, 3, 6], good) == (bad, [[1, 0], [1, 1], [1, 2]])   # beyond the table
    assert call([3, 3], [0, 3, 6], [[4], [1]]) == (bad, [[1, 0], [1, 1], [1, 2]])
    assert call([3, 3], [0, 3, 6], [[-1], [1]]) == (bad, [[1, 0], [1, 1], [1, 2]])
    assert call([3, 9], [0, 3, 9], good)[0] == bad                             # more rows than given
    assert call([3, 3], [3, 0, 6], good)[0] == bad                             # descending
    assert call([-3, 3], [0, 3, 6], good) == (bad, [[1, 0], [1, 1], [1, 2]])


# ------------------------------------------------------------ together, in use

def test_captured_step_serves_other_lengths_and_pages():
    """One captured append + decode step replays with other lengths, pages and
    values; a padding sequence joins in."""
    B, G, R, page, cols = 4, 2, 4, 16, 20
    gen = torch.Generator().manual_seed(21)
    kp, vp = (torch.randn(B * cols, page, G, 128, generator=gen).to(BF16).to(DEV) for _ in range(2))
    table = torch.arange(B * cols, dtype=torch.int32).reshape(B, cols).to(DEV)
    lens = torch.tensor([5, 17, 300, 0], dtype=torch.int32, device=DEV)
    q, k, v = (torch.randn(B, h, 128, generator=gen).to(BF16).to(DEV) for h in (G * R, G, G))
    f = (10000.0 ** (-torch.arange(64).float() / 64)).to(DEV)
    wa = M.new_paged_workspace(M.MSA_OP_PAGED_APPEND, table, page, G * R, G)
    wd = M.new_paged_workspace(M.MSA_OP_PAGED_DECODE, table, page, G * R, G)
    qo, out = torch.zeros_like(q), torch.zeros_like(q)
    lse = torch.zeros(B, G * R, device=DEV)

    def step():
        M.msa_paged_append(k, v, kp, vp, table, lens, q=q, q_out=qo, inv_freq=f, ws=wa)
        M.msa_paged_attn_decode(qo, kp, vp, table, lens, out=out, lse=lse, ws=wd)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        step()
        s.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            step()
    for n in ([5, 17, 300, 0], [320, 1, 0, 16], [31, 32, 33, 257]):
        for t in (q, k, v):
            t.copy_(torch.randn(t.shape, generator=gen).to(BF16))
        lens.copy_(torch.tensor(n, dtype=torch.int32))
        table.copy_(torch.randperm(B * cols, generator=gen).to(torch.int32).reshape(B, cols))
        kc, vc = kp.clone(), vp.clone()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        qe = torch.zeros_like(q)
        qe[:] = qo                                # (a padding row keeps what it held)
        M.msa_paged_append(k, v, kc, vc, table, lens, q=q, q_out=qe, inv_freq=f)
        assert torch.equal(kc, kp) and torch.equal(vc, vp) and torch.equal(qe, qo)
        c = {"table": table, "k": kp, "v": vp, "ks": None, "vs": None}
        check_decode(c, qo, n, out, lse)
    assert M.msa_read_status(wa) == M.MSA_OK and M.msa_read_status(wd) == M.MSA_OK


def test_two_streams_at_once_with_their_own_workspaces():
    lens = [4000, 1, 900, 2500]
    c = make_cache(lens, 4, 64, False, seed=31)
    q = torch.randn(4, 16, 128, generator=torch.Generator().manual_seed(1)).to(BF16).to(DEV)
    t = torch.tensor(lens, dtype=torch.int32, device=DEV)
    want = M.msa_paged_attn_decode(q, c["k"], c["v"], c["table"], t)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    ws = [M.new_paged_workspace(M.MSA_OP_PAGED_DECODE, c["table"], 64, 16, 4) for _ in range(2)]
    outs = [[torch.zeros_like(q) for _ in range(20)] for _ in range(2)]
    torch.cuda.synchronize()
    for i in range(20):
        for x, s in enumerate(streams):
            M.msa_paged_attn_decode(q, c["k"], c["v"], c["table"], t, out=outs[x][i], ws=ws[x], stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for x in outs for o in x)


@pytest.mark.parametrize("fp8", [False, True])
def test_pages_behind_four_billion_values(fp8):
    """A pool of more than 2^32 values: the last pages are written and read."""
    G, page, H = 8, 256, 16
    num = (1 << 32) // (page * G * 128) + 9
    kind = torch.uint8 if fp8 else BF16
    kp, vp = (torch.zeros(num, page, G, 128, dtype=kind, device=DEV) for _ in range(2))
    ks, vs = (torch.zeros(num, page, G, device=DEV) if fp8 else None for _ in range(2))
    small = [torch.zeros(9, page, G, 128, dtype=kind, device=DEV) for _ in range(2)]
    ss = [torch.zeros(9, page, G, device=DEV) if fp8 else None for _ in range(2)]
    n = 700
    gen = torch.Generator().manual_seed(3)
    k, v = (torch.randn(n, G, 128, generator=gen).to(BF16).to(DEV) for _ in range(2))
    q = torch.randn(1, H, 128, generator=gen).to(BF16).to(DEV)
    lens = torch.tensor([n], dtype=torch.int32, device=DEV)
    cu = torch.tensor([0, n], dtype=torch.int32, device=DEV)
    outs = []
    for a, b, sa, sb, first in ((kp, vp, ks, vs, num - 9), (*small, *ss, 0)):
        table = torch.tensor([[first + 8, first + 3, first + 5]], dtype=torch.int32, device=DEV)
        M.msa_paged_append(k, v, a, b, table, lens, cu_new=cu, k_scale=sa, v_scale=sb)
        outs.append(M.msa_paged_attn_decode(q, a, b, table, lens, k_scale=sa, v_scale=sb))
    torch.cuda.synchronize()
    assert torch.equal(kp[num - 9:], small[0]) and torch.equal(vp[num - 9:], small[1])
    assert not kp[:16].any()
    assert torch.equal(*outs)


@pytest.mark.parametrize("scales", ["wide", "signed", "zero"])
def test_decode_fp8_scales_of_any_size(scales):
    """Scales from 1e-12 to 1e12 beside each other, negative ones, zeros."""
    lens = [300, 33]
    c = make_cache(lens, 2, 16, True, seed=41)
    gen = torch.Generator().manual_seed(5)
    s = torch.rand(c["vs"].shape, generator=gen) + 0.5
    if scales == "wide":
        s = s * 10.0 ** (24 * torch.rand(s.shape, generator=gen) - 12)
    elif scales == "signed":
        s = s * (2 * torch.randint(0, 2, s.shape, generator=gen) - 1)
    else:
        s = s * torch.randint(0, 2, s.shape, generator=gen)
    c["vs"] = torch.where(c["own"][..., None].to(DEV), s.to(DEV), float("nan"))
    q = torch.randn(2, 16, 128, generator=gen).to(BF16).to(DEV)
    out, lse = decode(c, q, lens)
    check_decode(c, q, lens, out, lse)
    if scales == "zero":
        c["vs"] = torch.where(c["own"][..., None].to(DEV), torch.zeros_like(c["vs"]), float("nan"))
        out, _ = decode(c, q, lens)
        assert (out == 0).all()


def test_append_fp8_rows_of_tiny_and_large_values():
    """Rows whose scale is subnormal, or whose values end at the type's top."""
    G, page = 4, 16
    k = torch.zeros(1, G, 128, dtype=BF16)
    k[0, 0, :64] = 1e-40                 # subnormal values, zeros beside them
    k[0, 1] = (torch.linspace(-1, 1, 128) * 3.3e38).to(BF16)
    k[0, 2] = torch.linspace(-1e-36, 1e-36, 128).to(BF16)
    k[0, 3, 5] = 2.0 ** -133             # the smallest subnormal
    assert torch.isfinite(k).all()
    k = k.to(DEV)
    kp, vp = (torch.zeros(2, page, G, 128, dtype=torch.uint8, device=DEV) for _ in range(2))
    ks, vs = (torch.zeros(2, page, G, device=DEV) for _ in range(2))
    table = torch.tensor([[1]], dtype=torch.int32, device=DEV)
    M.msa_paged_append(k, k, kp, vp, table, torch.tensor([4], dtype=torch.int32, device=DEV), k_scale=ks, v_scale=vs)
    codes = kp[1, 3].cpu()
    got = codes.view(torch.float8_e4m3fn).float()
    assert torch.isfinite(got).all()
    want = f64(k[0])
    rel = got.double().numpy() / 448 * np.abs(want).max(-1, keepdims=True)
    # half a step of a code (2^-4 of a normal one), and the largest is met
    assert (np.abs(rel - want) <= np.maximum(2.0 ** -4 * np.abs(want), 2.0 ** -9 * np.abs(want).max(-1, keepdims=True))).all()
    assert (got.abs().amax(-1) == 448).all()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("G,R,lens", [(2, 4, [40, 900, 70]), (1, 16, [3, 5000]), (4, 8, [20000, 300, 9000] + [1] * 30)])
def test_decode_nan_stays_with_its_head(G, R, lens, fp8):
    """Token 17 of sequence 1 holds a NaN key (head 0) or value (the last
    head): that head's results are NaN, all others keep their bits."""
    c = make_cache(lens, G, 16, fp8, seed=G)
    q = torch.randn(len(lens), G * R, 128, generator=torch.Generator().manual_seed(4)).to(BF16).to(DEV)
    out, lse = decode(c, q, lens)
    at = (int(c["table"][1, 1]), 1)
    for x, g in (("k", 0), ("v", G - 1)):
        bad = dict(c)
        bad[x] = c[x].clone()
        bad[x][at[0], at[1], g] = 0x7F if fp8 else float("nan")
        o, ls = decode(bad, q, lens)
        hit = torch.zeros(len(lens), G * R, dtype=torch.bool, device=DEV)
        hit[1, g * R:(g + 1) * R] = True
        assert torch.isnan(o[hit]).all() and torch.equal(o[~hit], out[~hit])
        if x == "k":
            assert torch.isnan(ls[hit]).all()
        else:
            assert torch.equal(ls[hit], lse[hit])
        assert torch.equal(ls[~hit], lse[~hit])


def test_append_fp8_codes_are_those_of_the_quotient():
    """Every bf16 significand as a row's largest value, against every other one
    at twelve powers of two: each code is that of x / scale (92 of these
    quotients lie so near the middle of two codes that x times 1 / scale
    would get the other one)."""
    page, m = 64, torch.arange(128.0, 256.0)
    x = torch.stack([torch.minimum(m[None] * 2.0 ** -j, m[:, None]) for j in range(12)])   # [12, largest, 128]
    x[..., 127] = m                               # (255 2^-j gives way to the largest)
    n = 12 * 128 // 4
    k = x.view(n, 4, 128).to(BF16)
    assert torch.equal(k.float(), x.view(n, 4, 128))
    kp, vp = (torch.zeros(n // page, page, 4, 128, dtype=torch.uint8, device=DEV) for _ in range(2))
    ks, vs = (torch.zeros(n // page, page, 4, device=DEV) for _ in range(2))
    table = torch.arange(n // page, dtype=torch.int32, device=DEV).reshape(1, -1)
    M.msa_paged_append(k.to(DEV), -k.to(DEV), kp, vp, table, torch.tensor([n], dtype=torch.int32, device=DEV),
                       cu_new=torch.tensor([0, n], dtype=torch.int32, device=DEV), k_scale=ks, v_scale=vs)
    scale = k.float().abs().amax(-1) / 448
    want = (k.float() / scale[..., None]).to(torch.float8_e4m3fn).float()
    for codes, sc, sign in ((kp, ks, 1.0), (vp, vs, -1.0)):
        assert torch.equal(sc.view(n, 4).cpu(), scale)
        got = codes.view(n, 4, 128).cpu().view(torch.float8_e4m3fn).float()
        assert torch.equal(got, sign * want)


@pytest.mark.parametrize("cols", [20, 300])       # the one-launch form and the split one
@pytest.mark.parametrize("G,R", [(2, 4), (2, 8), (2, 1), (2, 16)])
@pytest.mark.parametrize("gain", [1e-9, 1e-5, 1e-35, 1e7, 1e35])
def test_decode_fp8_queries_of_any_size(gain, G, R, cols):
    """Queries far under and over what f16 holds, against keys whose scales
    bring the scores back (KV head 0); beside them (1) heads of every size;
    and elements of every size within a row."""
    lens = [300, 33]
    c = make_cache(lens, G, 16, True, seed=51, cols=cols)
    c["ks"][..., 0] /= gain
    q = torch.randn(2, G, R, 128, generator=torch.Generator().manual_seed(6))
    q[1] *= 2.0 ** -torch.arange(128).div(8, rounding_mode="floor")
    q[:, 0] *= gain
    q[0, 1] *= 2.0 ** -(3.0 * torch.arange(R))[:, None]
    q = q.view(2, G * R, 128).to(BF16).to(DEV)
    out, lse = decode(c, q, lens)
    check_decode(c, q, lens, out, lse)


@pytest.mark.parametrize("G,R,lens,cols", [(2, 4, [300, 33], 20), (2, 16, [300, 33], 20), (1, 4, [5000, 70], 330),
                                           (1, 16, [5000, 70], 330), (1, 8, [90000], 5630)])
def test_decode_fp8_tail_behind_sinks(G, R, lens, cols):
    """Every sixteenth key takes nearly all of the weight and has a value of
    zero: what comes out is the others' share, 2^-26 of it each."""
    c = make_cache(lens, G, 16, True, seed=52, cols=cols)
    gen = torch.Generator().manual_seed(7)
    own, shape = c["own"], c["k"].shape
    k0 = torch.randint(-1, 2, shape[:3], generator=gen).float() / 4
    v = torch.randn(shape, generator=gen).abs() + 0.5
    sink = torch.zeros(shape[:3], dtype=torch.bool)
    sink[:, 3] = True
    k0[sink], v[sink] = 18.0, 0.0                  # e^-18 = 2^-25.97
    k = c["k"].cpu().view(torch.float8_e4m3fn).float()
    k[..., 0] = k0
    for x, t in (("k", k), ("v", v)):
        codes = t.to(torch.float8_e4m3fn).view(torch.uint8)
        codes[~own] = 0x7F
        c[x] = codes.to(DEV)
    c["ks"] = torch.where(own[..., None], 1.0, float("nan")).expand(shape[:3]).contiguous().to(DEV)
    q = torch.zeros(len(lens), G * R, 128, device=DEV, dtype=BF16)
    q[..., 0] = 1.0
    out, lse = decode(c, q, lens, scale=1.0)
    check_decode(c, q, lens, out, lse, scale=1.0)
    assert (out[0] > 0).all()


def test_bad_pages_and_lengths_without_a_workspace_give_zeros():
    """A call that allocates its results and its workspace leaves nothing of
    older memory in rows that it skips."""
    junk = [torch.full((2 ** i,), 7.0, dtype=BF16, device=DEV) for i in range(6, 16) for _ in range(3)]
    del junk
    k = torch.ones(4, 1, 128, dtype=BF16, device=DEV)
    pages = [torch.zeros(4, 16, 1, 128, dtype=BF16, device=DEV) for _ in range(2)]
    table = torch.tensor([[0], [9]], dtype=torch.int32, device=DEV)
    n = torch.tensor([2, 2], dtype=torch.int32, device=DEV)
    cu = torch.tensor([0, 2, 4], dtype=torch.int32, device=DEV)
    q = torch.ones(4, 4, 128, dtype=BF16, device=DEV)
    out = M.msa_paged_append(k, k, *pages, table, n, cu_new=cu, q=q)
    assert (out[:2] == 1).all() and (out[2:] == 0).all()


@pytest.mark.parametrize("fp8", [False, True])
def test_decode_runs_that_start_behind_the_first_hundred_sequences(fp8):
    """200 sequences, long ones on both sides of the 128 whose tiles are summed
    at once, empty ones between: runs begin in the second lot and cross it."""
    rng = np.random.default_rng(8)
    lens = rng.integers(0, 40, 200).tolist()
    for b, n in ((3, 5000), (100, 2100), (126, 3000), (127, 0), (128, 4100), (129, 0), (150, 6000), (198, 900), (199, 0)):
        lens[b] = n
    c = make_cache(lens, 2, 16, fp8, seed=53)
    q = torch.randn(200, 8, 128, generator=torch.Generator().manual_seed(8)).to(BF16).to(DEV)
    ws = M.new_paged_workspace(M.MSA_OP_PAGED_DECODE, c["table"], 16, 8, 2)
    out, lse = decode(c, q, lens, ws=ws)
    check_decode(c, q, lens, out, lse)
    again, _ = decode(c, q, lens, ws=ws)
    assert torch.equal(out, again)
    assert M.msa_read_status(ws) == M.MSA_OK


@pytest.mark.parametrize("lens,G,R,cols", [([300, 33, 1], 2, 4, 20), ([300, 33, 2], 1, 16, 20), ([9000, 700], 2, 8, 600),
                                           ([9000, 700], 1, 16, 600), ([5000], 1, 1, 400)])
def test_decode_bf16_rounds_nothing_but_its_results(lens, G, R, cols):
    """The weights enter their product in two bf16 terms, so what they lose is
    a rounding of a rounding's rest, 2^-16 of them; the result is rounded once."""
    c = make_cache(lens, G, 16, False, seed=54, cols=cols)
    q = torch.randn(len(lens), G * R, 128, generator=torch.Generator().manual_seed(9)).to(BF16).to(DEV)
    out = f64(decode(c, q, lens)[0])
    for b, n in enumerate(lens):
        k, v = gathered(c, "k", b, n), gathered(c, "v", b, n)
        for h in range(G * R):
            ref, _, p, _, dz = O.attend(f64(q[b, h])[None], k[:, h // R], v[:, h // R], 128 ** -0.5, [n])
            tol = O.U * np.abs(ref) + (2.0 ** -16 + 2 * (dz + 2.0 ** -20))[:, None] * (p @ np.abs(v[:, h // R]))
            err = np.abs(out[b, h] - ref[0])
            assert (err <= tol[0]).all(), (b, h, (err - tol[0]).max())


@pytest.mark.parametrize("cols", [60, 300])
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("R", [1, 4, 16])
def test_decode_nan_in_a_query_stays_with_its_head(R, fp8, cols):
    lens = [40, 900, 7]
    c = make_cache(lens, 2, 16, fp8, seed=55, cols=cols)
    q = torch.randn(3, 2 * R, 128, generator=torch.Generator().manual_seed(4)).to(BF16).to(DEV)
    out, lse = decode(c, q, lens)
    hit = torch.zeros(3, 2 * R, dtype=torch.bool, device=DEV)
    for b, h, d, x in ((0, R, 5, "nan"), (1, 0, 127, "nan"), (2, 2 * R - 1, 64, "inf")):
        q[b, h, d] = float(x)
        hit[b, h] = True
    o, ls = decode(c, q, lens)
    assert torch.isnan(o[hit][:2]).all() and torch.isnan(ls[hit][:2]).all()
    assert torch.equal(o[~hit], out[~hit]) and torch.equal(ls[~hit], lse[~hit])


@pytest.mark.parametrize("cols", [60, 300])
@pytest.mark.parametrize("R", [1, 4, 8, 16])
def test_decode_infinite_value_stays_in_its_dim(R, cols):
    lens = [40, 900, 7]
    c = make_cache(lens, 2, 16, False, seed=56, cols=cols)
    q = torch.randn(3, 2 * R, 128, generator=torch.Generator().manual_seed(4)).to(BF16).to(DEV)
    out, lse = decode(c, q, lens)
    for b, t, g, d, x in ((0, 17, 1, 5, "inf"), (1, 899, 0, 127, "-inf")):
        c["v"][c["table"][b, t // 16].long(), t % 16, g, d] = float(x)
    o, ls = decode(c, q, lens)
    hit = torch.zeros_like(out, dtype=torch.bool)
    hit[0, R:, 5], hit[1, :R, 127] = True, True
    assert torch.equal(o[~hit], out[~hit]) and torch.equal(ls, lse)
    if R <= 8:
        assert (o[0, R:, 5] == float("inf")).all() and (o[1, :R, 127] == -float("inf")).all()
    else:
        assert not torch.isfinite(o[hit]).any()
