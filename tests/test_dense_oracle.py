"""CPU pins of the dense oracle against torch in 64 bits, and the refusals
and host-side checks of the paged and packed entry points."""
import ctypes
import math

import numpy as np
import pytest
import torch

import block_sparse_long_08_b200.msa as M
import oracle.dense_oracle as O
from tests.test_binding_checks import _refused, _short, stub  # noqa: F401

BF16 = torch.bfloat16


def _packed(lens_q, lens_k, H, G, seed=0, d=16):
    gen = torch.Generator().manual_seed(seed)
    q = torch.randn(sum(lens_q), H, d, dtype=torch.float64, generator=gen)
    k, v = (torch.randn(sum(lens_k), G, d, dtype=torch.float64, generator=gen) for _ in range(2))
    return q, k, v, np.cumsum([0] + lens_q), np.cumsum([0] + lens_k)


@pytest.mark.parametrize("lens_q,lens_k", [([5, 1, 7], [5, 1, 7]), ([3, 4], [9, 4]), ([6], [2]),
                                           ([0, 3, 2], [4, 3, 0])])
def test_dense_oracle_matches_torch(lens_q, lens_k):
    H, G = 4, 2
    q, k, v, cq, ck = _packed(lens_q, lens_k, H, G)
    q, k, v = (x.requires_grad_() for x in (q, k, v))
    dout = torch.randn(q.shape, dtype=torch.float64, generator=torch.Generator().manual_seed(9))
    outs = []
    for b in range(len(lens_q)):
        qi, ki, vi = q[cq[b]:cq[b + 1]], k[ck[b]:ck[b + 1]], v[ck[b]:ck[b + 1]]
        n, m = lens_q[b], lens_k[b]
        mask = torch.ones(n, m, dtype=torch.bool).tril(m - n)
        z = torch.einsum("nhd,mhd->hnm", qi, ki.repeat_interleave(H // G, 1)) / math.sqrt(q.shape[2])
        z = z.masked_fill(~mask, -1e300)
        p = torch.softmax(z, -1) * mask if m else z
        outs.append(torch.einsum("hnm,mhd->nhd", p, vi.repeat_interleave(H // G, 1)))
    want = torch.cat(outs)
    (want * dout).sum().backward()
    a = [x.detach().numpy() for x in (q, k, v)]
    out, lse, _, _ = O.dense(*a, cq, ck)
    assert np.abs(out - want.detach().numpy()).max() < 1e-12
    grads, _ = O.dense_backward(*a, dout.numpy(), cq, ck)
    for n, x in (("dq", q), ("dk", k), ("dv", v)):
        assert np.abs(grads[n] - x.grad.numpy()).max() < 1e-12, n


def test_dense_gradients_against_differences():
    q, k, v, cq, ck = _packed([4, 3], [6, 3], 2, 1, seed=3)
    a = {"q": q.numpy(), "k": k.numpy(), "v": v.numpy()}
    rng = np.random.default_rng(0)
    dout = rng.standard_normal(q.shape)
    grads, _ = O.dense_backward(a["q"], a["k"], a["v"], dout, cq, ck)
    for n in a:
        way = rng.standard_normal(a[n].shape)

        def loss(h):
            b = dict(a)
            b[n] = a[n] + h * way
            return (O.dense(b["q"], b["k"], b["v"], cq, ck)[0] * dout).sum()
        num = (loss(1e-5) - loss(-1e-5)) / 2e-5
        assert abs(num - (grads["d" + n] * way).sum()) < 1e-7


def test_rotation_keeps_lengths_and_relative_angles():
    rng = np.random.default_rng(1)
    x = rng.standard_normal((2, 1, 32))
    f = 10000.0 ** (-np.arange(16) / 16)
    for inter in (False, True):
        for far in (0, 12345):
            y = O.rotate(x, [3 + far, 7 + far], f, 32, inter)
            assert np.allclose((y ** 2).sum(-1), (x ** 2).sum(-1))
            near = O.rotate(x, [3, 7], f, 32, inter)
            assert np.isclose((y[0] * y[1]).sum(), (near[0] * near[1]).sum())
        z = O.rotate(x, [5, 5], f[:4], 8, inter)
        assert np.array_equal(z[..., 8:], x[..., 8:]) and not np.allclose(z[..., :8], x[..., :8])


# ------------------------------------------------------------- refusals (host)

def _cache(page=64, num=8, cols=4, k=4096, scales=False):
    return M.msa_paged_cache(k, 4096, 4096 if scales else None, None, 4096, num, page, cols)


OK = ctypes.c_void_p(4096)


def _append(p, c, n=2, cu=None, rot=0, q=None, q_out=None, ws=OK, ws_bytes=1 << 20, k=OK):
    return M.lib().msa_paged_append(ctypes.byref(p), ctypes.byref(c), n, q, k, OK, cu, OK, OK, rot, 0,
                                    q_out, None, ws, ws_bytes, None)


def test_append_refusals():
    p = M.make_params(2, 256, 8, 2)
    bad = ctypes.c_void_p(4100)
    for rc, code in [
            (_append(p, _cache(page=48)), M.MSA_ERR_UNSUPPORTED),
            (_append(p, _cache(page=512)), M.MSA_ERR_UNSUPPORTED),
            (_append(p, _cache(cols=3)), M.MSA_ERR_INVALID_ARG),       # L beyond the table
            (_append(p, _cache(scales=True)), M.MSA_ERR_INVALID_ARG),  # k_scale alone
            (_append(p, _cache(k=4100)), M.MSA_ERR_INVALID_ARG),
            (_append(p, _cache(num=-1)), M.MSA_ERR_INVALID_ARG),
            (_append(p, _cache(), n=3), M.MSA_ERR_INVALID_ARG),        # rows != B without cu_new
            (_append(p, _cache(), n=-1), M.MSA_ERR_INVALID_ARG),
            (_append(p, _cache(), rot=24), M.MSA_ERR_UNSUPPORTED),
            (_append(p, _cache(), rot=144), M.MSA_ERR_UNSUPPORTED),
            (_append(p, _cache(), q=OK), M.MSA_ERR_INVALID_ARG),       # q without q_out
            (_append(p, _cache(), k=bad), M.MSA_ERR_INVALID_ARG),
            (_append(p, _cache(), k=None), M.MSA_ERR_INVALID_ARG),
            (_append(p, _cache(), ws_bytes=8), M.MSA_ERR_WORKSPACE),
            (_append(p, _cache(), ws=None), M.MSA_ERR_WORKSPACE)]:
        assert rc == code, M.msa_last_error()
    for field, value, code in [("H", 6, M.MSA_ERR_UNSUPPORTED), ("G", 3, M.MSA_ERR_INVALID_ARG),
                               ("d", 64, M.MSA_ERR_UNSUPPORTED), ("B", -1, M.MSA_ERR_INVALID_ARG),
                               ("scale", -1.0, M.MSA_ERR_INVALID_ARG), ("H", 2048, M.MSA_ERR_UNSUPPORTED)]:
        q = M.make_params(2, 256, 8, 2)
        setattr(q, field, value)
        assert _append(q, _cache()) == code
        assert M.lib().msa_workspace_bytes(ctypes.byref(q), M.MSA_OP_PAGED_DECODE) == 0
    assert _append(M.make_params(0, 256, 8, 2), _cache(), n=0) == M.MSA_OK


def test_decode_refusals():
    def call(p, c=None, q=OK, lens=OK, out=OK, lse=None, ws_bytes=1 << 30):
        c = c or _cache()
        return M.lib().msa_paged_attn_decode(ctypes.byref(p), ctypes.byref(c), q, lens, out, lse, OK,
                                             ws_bytes, None)
    p = M.make_params(2, 256, 8, 2)
    assert call(p, _cache(page=8)) == M.MSA_ERR_UNSUPPORTED
    assert call(p, _cache(cols=1)) == M.MSA_ERR_INVALID_ARG
    assert call(p, q=None) == M.MSA_ERR_INVALID_ARG
    assert call(p, lens=None) == M.MSA_ERR_INVALID_ARG
    assert call(p, out=ctypes.c_void_p(4104)) == M.MSA_ERR_INVALID_ARG
    assert call(p, lse=ctypes.c_void_p(4098)) == M.MSA_ERR_INVALID_ARG
    assert call(p, ws_bytes=16) == M.MSA_ERR_WORKSPACE
    assert call(M.make_params(0, 256, 8, 2)) == M.MSA_OK
    # neither G <= 8 nor B * L <= 2^26 is asked for here
    assert M.msa_workspace_bytes(M.make_params(512, 1 << 20, 64, 32), M.MSA_OP_PAGED_DECODE) > 0


def test_dense_refusals():
    def fwd(p, nq=10, nk=10, q=OK, cu=OK, ws_bytes=1 << 30, lse=None):
        return M.lib().msa_dense_attn_varlen(ctypes.byref(p), nq, nk, q, OK, OK, cu, OK, OK, lse, OK,
                                             ws_bytes, None)

    def bwd(p, lse=OK, dq=OK, dout=OK, ws_bytes=1 << 30):
        return M.lib().msa_dense_attn_varlen_backward(ctypes.byref(p), 10, 10, OK, OK, OK, OK, lse, dout,
                                                      OK, OK, dq, OK, OK, OK, ws_bytes, None)
    p = M.make_params(2, 10, 8, 2)
    assert fwd(p, nq=11) == M.MSA_ERR_INVALID_ARG       # more rows than p->L
    assert fwd(p, nk=-1) == M.MSA_ERR_INVALID_ARG
    assert fwd(p, q=None) == M.MSA_ERR_INVALID_ARG
    assert fwd(p, q=ctypes.c_void_p(4104)) == M.MSA_ERR_INVALID_ARG
    assert fwd(p, cu=None) == M.MSA_ERR_INVALID_ARG
    assert fwd(p, lse=ctypes.c_void_p(4097)) == M.MSA_ERR_INVALID_ARG
    assert fwd(p, ws_bytes=100) == M.MSA_ERR_WORKSPACE
    assert bwd(p, lse=None) == M.MSA_ERR_INVALID_ARG
    assert bwd(p, dq=ctypes.c_void_p(4104)) == M.MSA_ERR_INVALID_ARG
    assert bwd(p, dout=None) == M.MSA_ERR_INVALID_ARG
    assert bwd(p, ws_bytes=100) == M.MSA_ERR_WORKSPACE
    p.G = 3
    assert fwd(p) == M.MSA_ERR_INVALID_ARG
    assert fwd(M.make_params(0, 10, 8, 2)) == M.MSA_OK
    assert fwd(M.make_params(2, 10, 8, 2), nq=0, q=None) == M.MSA_OK


def test_binding_paged(stub):  # noqa: F811
    B, H, G, d = 3, 8, 2, 128
    q, k = torch.zeros(B, H, d, dtype=BF16), torch.zeros(B, G, d, dtype=BF16)
    pages = torch.zeros(9, 32, G, d, dtype=BF16)
    table = torch.zeros(B, 3, dtype=torch.int32)
    lens = torch.ones(B, dtype=torch.int32)
    f = torch.ones(64)
    assert M.msa_paged_append(k, k, pages, pages, table, lens, q=q, inv_freq=f).shape == q.shape
    assert M.msa_paged_append(k, k, pages, pages, table, lens) is None
    out, lse = M.msa_paged_attn_decode(q, pages, pages, table, lens, want_lse=True)
    assert out.shape == q.shape and lse.shape == (B, H)
    codes, sc = pages.to(torch.uint8), torch.ones(9, 32, G)
    M.msa_paged_append(k, k, codes, codes, table, lens, k_scale=sc, v_scale=sc)
    M.msa_paged_attn_decode(q, codes, codes, table, lens, k_scale=sc, v_scale=sc)
    assert stub.calls == ["msa_paged_append", "msa_paged_append", "msa_paged_attn_decode",
                          "msa_paged_append", "msa_paged_attn_decode"]
    ap, de = M.msa_paged_append, M.msa_paged_attn_decode
    _refused(stub, ap, k, _short(k), pages, pages, table, lens)
    _refused(stub, ap, k, k, pages, pages, table, _short(lens))
    _refused(stub, ap, k, k, pages, _short(pages), table, lens, match="must be")
    _refused(stub, ap, k, k, codes, codes, table, lens, match="must be torch.bfloat16")
    _refused(stub, ap, k, k, codes, codes, table, lens, k_scale=sc, match="both")
    _refused(stub, ap, k, k, codes, codes, table, lens, k_scale=sc, v_scale=_short(sc))
    _refused(stub, ap, k[:2], k[:2], pages, pages, table, lens, match="cu_new")
    _refused(stub, ap, k, k, pages, pages, table, lens, cu_new=lens)
    _refused(stub, ap, k, k, pages, pages, table, lens, rot_dim=64, match="inv_freq")
    _refused(stub, ap, k, k, pages, pages, table, lens, rot_dim=128, inv_freq=f[:8])
    _refused(stub, ap, k, k, pages, pages, table, lens, q_out=q, match="without q")
    _refused(stub, ap, k, k, pages, pages, table, lens, q=q, q_out=_short(q))
    _refused(stub, ap, k, k, pages, pages, table.long(), lens, match="must be torch.int32")
    _refused(stub, ap, k, k, pages[:, :, :1].contiguous(), pages[:, :, :1].contiguous(), table, lens,
             match="KV heads")
    _refused(stub, de, q, pages, pages, table[:2].contiguous(), lens, match="page_table rows")
    _refused(stub, de, q, pages, pages, table, _short(lens))
    _refused(stub, de, q, pages, pages, table, lens, out=_short(q))
    _refused(stub, de, q, pages, pages, table, lens, lse=torch.zeros(B, H - 1))
    _refused(stub, de, q, pages.transpose(0, 1), pages.transpose(0, 1), table, lens, match="contiguous")


def test_binding_dense(stub):  # noqa: F811
    q, k = torch.zeros(10, 8, 128, dtype=BF16), torch.zeros(12, 2, 128, dtype=BF16)
    cq, ck = torch.tensor([0, 4, 10], dtype=torch.int32), torch.tensor([0, 6, 12], dtype=torch.int32)
    out, lse = M.msa_dense_attn_varlen(q, k, k, cq, ck, want_lse=True)
    dq, dk, dv = M.msa_dense_attn_varlen_backward(q, k, k, out, lse, out, cq, ck)
    assert dq.shape == q.shape and dk.shape == dv.shape == k.shape
    assert stub.calls == ["msa_dense_attn_varlen", "msa_dense_attn_varlen_backward"]
    fwd, bwd = M.msa_dense_attn_varlen, M.msa_dense_attn_varlen_backward
    _refused(stub, fwd, q, k, _short(k), cq, ck)
    _refused(stub, fwd, q, k, k, cq, _short(ck))
    _refused(stub, fwd, q, k, k, cq.long(), ck, match="must be torch.int32")
    _refused(stub, fwd, q, k, k, cq, ck, out=_short(out))
    _refused(stub, fwd, q, k, k, cq, ck, lse=_short(lse))
    _refused(stub, bwd, q, k, k, out, _short(lse), out, cq, ck)
    _refused(stub, bwd, q, k, k, out, lse, _short(out), cq, ck)
    _refused(stub, bwd, q, k, k, out, lse, out, cq, ck, dk=_short(k))
    _refused(stub, bwd, q, k, k, out, lse, out, cq, ck, dq=out.float(), match="must be torch.bfloat16")


def test_binding_refuses_two_devices(stub):  # noqa: F811
    q, k = torch.zeros(4, 8, 128, dtype=BF16), torch.zeros(4, 2, 128, dtype=BF16)
    cu = torch.tensor([0, 4], dtype=torch.int32)
    _refused(stub, M.msa_dense_attn_varlen, q, k, k.to("meta"), cu, cu, match="is on meta")


def test_binding_refuses_rows_of_another_shape(stub):  # noqa: F811
    """Enough elements in all, but not the rows the call would read."""
    q, k = torch.zeros(10, 8, 128, dtype=BF16), torch.zeros(12, 2, 128, dtype=BF16)
    cq, ck = torch.tensor([0, 10], dtype=torch.int32), torch.tensor([0, 12], dtype=torch.int32)
    out, lse = torch.zeros_like(q), torch.zeros(10, 8)
    wide, turned = torch.zeros(12, 2, 256, dtype=BF16), torch.zeros(8, 10, 128, dtype=BF16)
    fwd, bwd = M.msa_dense_attn_varlen, M.msa_dense_attn_varlen_backward
    _refused(stub, fwd, q, wide, wide, cq, ck, match="k must be")
    _refused(stub, fwd, q, k, wide, cq, ck, match="v must be")
    _refused(stub, fwd, q, k, k.reshape(12, 256), cq, ck, match="v must be")
    _refused(stub, bwd, q, k, k, out, lse, turned, cq, ck, match="dout must be")
    _refused(stub, bwd, q, k, k, turned, lse, out, cq, ck, match="out must be")
    pages, table = torch.zeros(9, 32, 2, 128, dtype=BF16), torch.zeros(3, 3, dtype=torch.int32)
    lens, k3 = torch.ones(3, dtype=torch.int32), torch.zeros(3, 2, 128, dtype=BF16)
    _refused(stub, M.msa_paged_append, k3, torch.zeros(3, 4, 128, dtype=BF16), pages, pages, table, lens,
             match="v must be")
    _refused(stub, M.msa_paged_append, k3, k3, pages, pages, table, lens, q=torch.zeros(3, 8, 256, dtype=BF16),
             match="q must be")
    _refused(stub, M.msa_paged_attn_decode, q[:3], pages[0], pages[0], table, lens, match="k_pages, v_pages must")


def test_backward_refuses_results_over_what_it_reads():
    """Two kernels run at once: no gradient may lie over an input of the other
    one, or over another gradient."""
    p = M.make_params(1, 10, 8, 2)
    big, small = 10 * 8 * 128 * 2, 10 * 2 * 128 * 2
    at = {n: (i + 1) << 20 for i, n in enumerate(("q", "k", "v", "out", "lse", "dout", "cq", "ck", "dq", "dk", "dv", "ws"))}

    def call(**kw):
        a = {n: ctypes.c_void_p(x) for n, x in {**at, **kw}.items()}
        return M.lib().msa_dense_attn_varlen_backward(
            ctypes.byref(p), 10, 10, a["q"], a["k"], a["v"], a["out"], a["lse"], a["dout"], a["cq"], a["ck"],
            a["dq"], a["dk"], a["dv"], a["ws"], 1 << 20, None)
    sizes = {"q": big, "dout": big, "k": small, "v": small, "dq": big, "dk": small, "dv": small}
    for res in ("dq", "dk", "dv"):
        for other in sizes:
            if other == res:
                continue
            for x in (at[other], at[other] + sizes[other] - 16, at[other] - sizes[res] + 16):
                assert call(**{res: x}) == M.MSA_ERR_INVALID_ARG, (res, other)
                assert "overlap" in M.msa_last_error()


def test_binding_allocates_zeros_where_rows_may_be_skipped(stub, monkeypatch):  # noqa: F811
    """Nothing of older memory in a result that the call allocates together
    with its workspace; a caller's buffers are left alone."""
    fill = torch.full
    monkeypatch.setattr(M.torch, "empty", lambda *a, **kw: fill(a[0] if len(a) == 1 else a, 7, **kw))
    monkeypatch.setattr(M.torch, "empty_like", lambda t, **kw: fill(t.shape, 7, dtype=t.dtype))
    q, k = torch.zeros(10, 8, 128, dtype=BF16), torch.zeros(12, 2, 128, dtype=BF16)
    cq, ck = torch.tensor([0, 4, 10], dtype=torch.int32), torch.tensor([0, 6, 12], dtype=torch.int32)
    res = M.msa_dense_attn_varlen(q, k, k, cq, ck, want_lse=True)
    res += M.msa_dense_attn_varlen_backward(q, k, k, q, res[1], q, cq, ck)
    pages, table = torch.zeros(9, 32, 2, 128, dtype=BF16), torch.zeros(3, 3, dtype=torch.int32)
    lens = torch.ones(3, dtype=torch.int32)
    res += (M.msa_paged_append(k[:3], k[:3], pages, pages, table, lens, q=q[:3]),)
    assert len(res) == 6 and all((t == 0).all() for t in res)
    mine = fill(q.shape, 3.0, dtype=BF16)
    assert M.msa_dense_attn_varlen(q, k, k, cq, ck, out=mine) is mine and (mine == 3).all()
