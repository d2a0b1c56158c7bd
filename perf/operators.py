"""The dense paged path's operators as a user's program calls them, with their
plain forms: what is measured and what the kernels' outputs are compared with.

    append    keys, values (and queries) of new tokens rotated by position,
              the keys and values written into a paged cache
    decode    one new token per sequence over a paged cache
    prompt    causal attention over packed prompts, the queries aligned to the
              end of their sequence's keys (a cached prefix may precede them)
    training  the same attention's forward and backward pass

A case is a dict of plain values.  The lengths of its sequences follow from
the case alone (`lengths`), so `work` knows them; inputs follow from the seed.
"""
import math
import random

import torch

own = False

D = 128            # head dim
BASE = 1.0e6       # base of the rotation's frequencies
DEV = "cuda"


# ------------------------------------------------------------------- cases

def listed():
    return [
        # one decode step's append: 64 running requests, one token each
        dict(name="append_step", op="append", B=64, lo=200, hi=2000, one=True, H=32, G=8, page=64, rot=128,
             inter=False, fp8=False, salt=1),
        # the prompts of an admitted batch, packed, 32K tokens
        dict(name="append_prompts", op="append", B=9, lo=1000, hi=6300, one=False, H=32, G=8, page=64, rot=128,
             inter=False, fp8=False, salt=2),
        # prompts into an 8-bit cache of small pages, half of each head rotated, neighbouring pairs
        dict(name="append_prompts_fp8", op="append", B=5, lo=500, hi=3001, one=False, H=16, G=4, page=16, rot=64,
             inter=True, fp8=True, salt=3),
        # a single interactive request: latency
        dict(name="decode_single", op="decode", B=1, lo=2047, hi=2047, H=8, G=2, page=64, fp8=False, salt=4),
        # a ragged serving batch at long context
        dict(name="decode_128k", op="decode", B=16, lo=65536, hi=131072, H=32, G=8, page=64, fp8=False, salt=5),
        # one request at a million tokens
        dict(name="decode_1m", op="decode", B=1, lo=1048575, hi=1048575, H=32, G=8, page=128, fp8=False, salt=6),
        # many short requests, 8-bit cache, small pages
        dict(name="decode_fp8", op="decode", B=96, lo=1, hi=16384, H=64, G=8, page=16, fp8=True, salt=7),
        # a few short prompts: latency
        dict(name="prompt_short", op="prompt", B=3, lo=5, hi=400, pre=0, H=8, G=2, salt=8),
        # prompts continued after cached prefixes
        dict(name="prompt_prefix", op="prompt", B=6, lo=300, hi=1900, pre=2000, H=32, G=8, salt=9),
        # one tensor-parallel shard of a 32K prompt
        dict(name="prompt_32k", op="prompt", B=1, lo=32768, hi=32768, pre=0, H=8, G=1, salt=10),
        # packed documents of a training batch
        dict(name="training_packed", op="training", B=7, lo=100, hi=1500, pre=0, H=16, G=4, salt=11),
        # one long training sequence
        dict(name="training_8k", op="training", B=1, lo=8192, hi=8192, pre=0, H=32, G=8, salt=12),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "decode", "prompt", "training"])
    r = rng.choice([1, 2, 4, 8, 16])
    g = rng.choice([1, 2, 4, 8])
    while g * r > 64:
        g //= 2
    case = dict(op=op, H=g * r, G=g, salt=rng.randrange(1 << 20))
    if op == "append":
        one = rng.random() < 0.4
        hi = _log(rng, 64, 2000 if one else 30000)
        case.update(B=_log(rng, 1, 128) if one else _log(rng, 1, max(1, 32768 // hi)), lo=rng.randint(1, hi), hi=hi, one=one,
                    page=rng.choice([16, 32, 64, 128, 256]), rot=rng.choice([0, 32, 64, 96, 128]),
                    inter=rng.random() < 0.5, fp8=rng.random() < 0.5)
    elif op == "decode":
        hi = _log(rng, 1, 200000)
        case.update(B=_log(rng, 1, max(1, min(128, 1000000 // hi))), lo=rng.randint(1, hi), hi=hi,
                    page=rng.choice([16, 32, 64, 128, 256]), fp8=rng.random() < 0.5)
    else:
        top = 8192 if op == "training" else 12000
        hi = _log(rng, 1, top)
        most = max(1, min(64, int(top * (32 / (g * r)) ** 0.5) // hi))
        case.update(B=_log(rng, 1, most), lo=rng.randint(1, hi), hi=hi,
                    pre=0)
        if rng.random() < 0.5:
            case["pre"] = _log(rng, 1, max(1, min(2000, top // case["B"])))
        while case["H"] > 32:
            case["H"], case["G"] = case["H"] // 2, max(1, case["G"] // 2)
    return case


def lengths(case):
    """(tokens of each sequence in the cache or among the keys, new ones among
    them): every sequence's lengths, from the case alone."""
    rng = random.Random(case["salt"])
    total, new = [], []
    for _ in range(case["B"]):
        n = rng.randint(case["lo"], case["hi"])
        if case["op"] == "append":
            before = n if case["one"] else rng.randint(0, 100)
            new.append(1 if case["one"] else n)
            total.append(before + new[-1])
        elif case["op"] == "decode":
            new.append(1)
            total.append(n)
        else:
            new.append(n)
            total.append(n + (rng.randint(0, case["pre"]) if case["pre"] else 0))
    return total, new


def _pairs(case):
    return sum(n * (t - n) + n * (n + 1) // 2 for t, n in zip(*lengths(case)))


def work(case):
    total, new = lengths(case)
    H, G, op = case["H"], case["G"], case["op"]
    nq, nk = sum(new), sum(total)
    if op == "append":
        stored = 2 * G * (D + 4) if case["fp8"] else 2 * G * D * 2
        return {"bytes": nq * (2 * H * D * 2 + 2 * G * D * 2 + stored), "flops": nq * (H + G) * case["rot"] * 3}
    if op == "decode":
        stored = 2 * G * (D + 4) if case["fp8"] else 2 * G * D * 2
        return {"bytes": nk * stored + 2 * nq * H * D * 2 + nq * H * 4, "flops": 4 * D * H * nk}
    rows = nq * H * (2 * D * 2 + 4) + 2 * nk * G * D * 2
    if op == "prompt":
        return {"bytes": rows, "flops": 4 * D * H * _pairs(case)}
    # the backward reads q, out, lse, dout, k, v and writes dq, dk, dv
    back = nq * H * (4 * D * 2 + 4) + 4 * nk * G * D * 2
    return {"bytes": rows + back, "flops": 14 * D * H * _pairs(case)}


# ------------------------------------------------------------------- inputs

def _starts(lens):
    return torch.tensor([0] + lens, dtype=torch.int64).cumsum(0).to(torch.int32).to(DEV)


def _pool(case, total, gen):
    """A page pool with the sequences' pages scattered over it, and the tables
    (-1 behind each sequence's last page)."""
    page, G = case["page"], case["G"]
    need = [-(-t // page) for t in total]
    pages = sum(need) + 3
    rng = random.Random(case["salt"] + 1)
    ids = list(range(pages))
    rng.shuffle(ids)
    table = torch.full((case["B"], max(need) + 1), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = torch.tensor(ids[at:at + n], dtype=torch.int32)
        at += n
    s = {"table": table.to(DEV)}
    shape = (pages, page, G, D)
    for x in ("k", "v"):
        if case["fp8"]:
            codes = torch.randint(0, 256, shape, dtype=torch.uint8, device=DEV, generator=gen)
            # codes of finite values within +-16: no exponent of 12 and more
            s[x + "_pages"] = torch.where((codes & 0x7F) < 0x58, codes, codes & 0xBF)
            s[x + "_scale"] = torch.rand(shape[:3], device=DEV, generator=gen) * 0.1 + 0.2
        else:
            s[x + "_pages"] = torch.randn(shape, device=DEV, generator=gen, dtype=torch.bfloat16)
            s[x + "_scale"] = None
    return s


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(int(seed))
    total, new = lengths(case)
    H, G, op = case["H"], case["G"], case["op"]
    nq, nk = sum(new), sum(total)

    def normal(*shape):
        return torch.randn(shape, device=DEV, generator=gen, dtype=torch.bfloat16)

    s = {"case": dict(case), "cache_lens": torch.tensor(total, dtype=torch.int32, device=DEV)}
    if op in ("append", "decode"):
        s.update(_pool(case, total, gen))
        s["q"] = normal(nq, H, D)
        s["out"] = torch.empty_like(s["q"])
        if op == "append":
            s["k"], s["v"] = normal(nq, G, D), normal(nq, G, D)
            s["cu"] = None if case["one"] else _starts(new)
            half = max(1, case["rot"] // 2)
            s["freq"] = (BASE ** (-torch.arange(half, dtype=torch.float64) / half)).float().to(DEV)
        else:
            s["lse"] = torch.empty((nq, H), device=DEV)
    else:
        s["q"], s["k"], s["v"] = normal(nq, H, D), normal(nk, G, D), normal(nk, G, D)
        s["cu_q"], s["cu_k"] = _starts(new), _starts(total)
        s["out"], s["lse"] = torch.empty_like(s["q"]), torch.empty((nq, H), device=DEV)
        if op == "training":
            s["dout"] = normal(nq, H, D)
            s["dq"], s["dk"], s["dv"] = (torch.empty_like(s[x]) for x in ("q", "k", "v"))
    # the status word and scratch that a program keeps between calls (asked for at the first call)
    s["ws"] = {}
    return s


# ------------------------------------------------------------------- passes

def run(state):
    op = state["case"]["op"]
    if own:
        return {"append": _own_append, "decode": _own_decode, "prompt": _own_prompt, "training": _own_training}[op](state)
    return {"append": _append, "decode": _decode, "prompt": _prompt, "training": _training}[op](state)


def _stored(s):
    """The cache as run() returns it: 8-bit codes as the values that they stand for, beside their scales."""
    if s["k_scale"] is None:
        return {"k_pages": s["k_pages"], "v_pages": s["v_pages"]}
    return {"k_pages": s["k_pages"].view(torch.float8_e4m3fn), "v_pages": s["v_pages"].view(torch.float8_e4m3fn),
            "k_scale": s["k_scale"], "v_scale": s["v_scale"]}


def _own_append(s):
    import block_sparse_long_08_b200.msa as M
    c = s["case"]
    if "append" not in s["ws"]:
        s["ws"]["append"] = M.new_paged_workspace(M.MSA_OP_PAGED_APPEND, s["table"], c["page"], c["H"], c["G"])
    M.msa_paged_append(s["k"], s["v"], s["k_pages"], s["v_pages"], s["table"], s["cache_lens"], cu_new=s["cu"],
                       q=s["q"], q_out=s["out"], inv_freq=s["freq"] if c["rot"] else None, rot_dim=c["rot"],
                       interleaved=c["inter"], k_scale=s["k_scale"], v_scale=s["v_scale"], ws=s["ws"]["append"])
    return {"q": s["out"], **_stored(s)}


def _own_decode(s):
    import block_sparse_long_08_b200.msa as M
    c = s["case"]
    if "decode" not in s["ws"]:
        s["ws"]["decode"] = M.new_paged_workspace(M.MSA_OP_PAGED_DECODE, s["table"], c["page"], c["H"], c["G"])
    M.msa_paged_attn_decode(s["q"], s["k_pages"], s["v_pages"], s["table"], s["cache_lens"], k_scale=s["k_scale"],
                            v_scale=s["v_scale"], out=s["out"], lse=s["lse"], ws=s["ws"]["decode"])
    return {"out": s["out"], "lse": s["lse"]}


def _own_forward(s):
    import block_sparse_long_08_b200.msa as M
    if "forward" not in s["ws"]:
        s["ws"]["forward"] = M.new_dense_workspace(M.MSA_OP_DENSE_VARLEN, s["q"], s["k"], s["case"]["B"])
    M.msa_dense_attn_varlen(s["q"], s["k"], s["v"], s["cu_q"], s["cu_k"], out=s["out"], lse=s["lse"],
                            ws=s["ws"]["forward"])


def _own_prompt(s):
    _own_forward(s)
    return {"out": s["out"], "lse": s["lse"]}


def _own_training(s):
    import block_sparse_long_08_b200.msa as M
    _own_forward(s)
    if "backward" not in s["ws"]:
        s["ws"]["backward"] = M.new_dense_workspace(M.MSA_OP_DENSE_VARLEN_BACKWARD, s["q"], s["k"], s["case"]["B"])
    M.msa_dense_attn_varlen_backward(s["q"], s["k"], s["v"], s["out"], s["lse"], s["dout"], s["cu_q"], s["cu_k"],
                                     dq=s["dq"], dk=s["dk"], dv=s["dv"], ws=s["ws"]["backward"])
    return {"out": s["out"], "dq": s["dq"], "dk": s["dk"], "dv": s["dv"]}


def _rows(s):
    """Sequence and position of each new token."""
    lens = s["cache_lens"].long()
    if s.get("cu") is None:
        return torch.arange(lens.numel(), device=DEV), lens - 1
    cu = s["cu"].long()
    at = torch.arange(s["k"].shape[0], device=DEV)
    b = torch.searchsorted(cu[1:].contiguous(), at, right=True)
    return b, lens[b] - (cu[b + 1] - at)


def _rotate(x, cos, sin, rot, inter):
    if rot == 0:
        return x
    cos, sin = cos[:, None], sin[:, None]
    y = x.clone()
    if inter:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y[..., 0:rot:2], y[..., 1:rot:2] = a * cos - b * sin, b * cos + a * sin
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y[..., :rot // 2], y[..., rot // 2:rot] = a * cos - b * sin, b * cos + a * sin
    return y


def _append(s):
    c = s["case"]
    b, pos = _rows(s)
    # angles in 64 bits: 32 lose them at far positions
    angle = pos.double()[:, None] * s["freq"].double()
    cos, sin = angle.cos().float(), angle.sin().float()
    s["out"].copy_(_rotate(s["q"].float(), cos, sin, c["rot"], c["inter"]))
    slot = s["table"][b, pos // c["page"]].long() * c["page"] + pos % c["page"]
    for x, y in (("k", _rotate(s["k"].float(), cos, sin, c["rot"], c["inter"])), ("v", s["v"].float())):
        if c["fp8"]:
            scale = y.abs().amax(-1) / 448
            scale = torch.where(scale > 0, scale, 1.0)
            codes = (y / scale[..., None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
            s[x + "_pages"].view(-1, c["G"], D)[slot] = codes
            s[x + "_scale"].view(-1, c["G"])[slot] = scale
        else:
            s[x + "_pages"].view(-1, c["G"], D)[slot] = y.to(torch.bfloat16)
    return {"q": s["out"], **_stored(s)}


def _cache(s, x):
    """[B, G, tokens of the longest sequence's pages, d] in 32 bits."""
    c = s["case"]
    need = -(-c["hi"] // c["page"])
    ids = s["table"][:, :need].long().clamp(min=0)
    y = s[x + "_pages"][ids]
    if c["fp8"]:
        y = y.view(torch.float8_e4m3fn).float() * s[x + "_scale"][ids][..., None]
    return y.view(c["B"], -1, c["G"], D).transpose(1, 2).float()


def _decode(s):
    c = s["case"]
    q = s["q"].float().view(c["B"], c["G"], -1, D)
    z = q @ _cache(s, "k").transpose(2, 3) / math.sqrt(D)
    behind = torch.arange(z.shape[3], device=DEV) >= s["cache_lens"].long()[:, None]
    z.masked_fill_(behind[:, None, None], -math.inf)
    top = z.amax(-1, keepdim=True)
    p = (z - top).exp()
    total = p.sum(-1, keepdim=True)
    out = p @ _cache(s, "v") / total
    return {"out": out.view(c["B"], c["H"], D).to(torch.bfloat16), "lse": (top + total.log()).view(c["B"], c["H"])}


def _probabilities(s):
    """P [H, nq, nk] before its division by the row sums, which come beside it with the logarithm of the whole."""
    c = s["case"]
    nq, nk, r = s["q"].shape[0], s["k"].shape[0], c["H"] // c["G"]
    cu_q, cu_k = s["cu_q"].long(), s["cu_k"].long()
    i, j = torch.arange(nq, device=DEV), torch.arange(nk, device=DEV)
    sq = torch.searchsorted(cu_q[1:].contiguous(), i, right=True)
    sk = torch.searchsorted(cu_k[1:].contiguous(), j, right=True)
    last = cu_k[sq + 1] - (cu_q[sq + 1] - i)      # the packed row of query i's own key
    hidden = (sk[None, :] != sq[:, None]) | (j[None, :] > last[:, None])
    q = s["q"].float().view(nq, c["G"], r, D).permute(1, 2, 0, 3).reshape(c["G"], r * nq, D)
    z = q @ s["k"].float().permute(1, 2, 0)
    z = z.view(c["H"], nq, nk).mul_(1 / math.sqrt(D)).masked_fill_(hidden[None], -math.inf)
    top = z.amax(-1, keepdim=True)
    z.sub_(top).exp_()
    total = z.sum(-1, keepdim=True)
    return z, total, (top + total.log())[..., 0].t().contiguous()


def _grouped(s, x, nq):
    """[nq, H, d] as [G, R nq, d]."""
    c = s["case"]
    return x.float().view(nq, c["G"], -1, D).permute(1, 2, 0, 3).reshape(c["G"], -1, D)


def _ungrouped(s, y, nq):
    c = s["case"]
    return y.view(c["G"], -1, nq, D).permute(2, 0, 1, 3).reshape(nq, c["H"], D)


def _prompt(s):
    nq = s["q"].shape[0]
    p, total, lse = _probabilities(s)
    out = p.view(s["case"]["G"], -1, p.shape[2]) @ s["v"].float().transpose(0, 1) / total.view(s["case"]["G"], -1, 1)
    return {"out": _ungrouped(s, out, nq).to(torch.bfloat16), "lse": lse}


def _training(s):
    c, nq = s["case"], s["q"].shape[0]
    p, total, _ = _probabilities(s)
    p = p.div_(total).view(c["G"], -1, p.shape[2])
    k, v = s["k"].float().transpose(0, 1), s["v"].float().transpose(0, 1)
    q, do = _grouped(s, s["q"], nq), _grouped(s, s["dout"], nq)
    out = p @ v
    dv = p.transpose(1, 2) @ do
    ds = (do @ v.transpose(1, 2)).sub_((do * out).sum(-1, keepdim=True)).mul_(p).mul_(1 / math.sqrt(D))
    return {"out": _ungrouped(s, out, nq).to(torch.bfloat16), "dq": _ungrouped(s, ds @ k, nq).to(torch.bfloat16),
            "dk": (ds.transpose(1, 2) @ q).transpose(0, 1).to(torch.bfloat16),
            "dv": dv.transpose(0, 1).to(torch.bfloat16)}


# ------------------------------------------------------------------- 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"append": _exact_append, "decode": _exact_decode, "prompt": _exact_dense, "training": _exact_dense}[case["op"]](s)


def _exact_append(s):
    c = s["case"]
    total, new = lengths(c)
    rot, half = c["rot"], c["rot"] // 2
    first = torch.arange(half, device=DEV) * (2 if c["inter"] else 1)
    second = first + (1 if c["inter"] else half)
    res = {"q": s["q"].double()}
    wide = {"k": s["k"].double(), "v": s["v"].double()}
    row = 0
    for b, (t, n) in enumerate(zip(total, new)):
        at = slice(row, row + n)
        row += n
        pos = torch.arange(t - n, t, device=DEV, dtype=torch.float64)
        if rot:
            turn = torch.polar(torch.ones((), dtype=torch.float64, device=DEV), pos[:, None, None] * s["freq"].double())
            for x in (res["q"], wide["k"]):
                z = torch.complex(x[at][..., first], x[at][..., second]) * turn
                y = x[at].clone()
                y[..., first], y[..., second] = z.real, z.imag
                x[at] = y
    for x in ("k", "v"):
        pages = s[x + "_pages"].view(torch.float8_e4m3fn).double() if c["fp8"] else s[x + "_pages"].double()
        scales = s[x + "_scale"].double() if c["fp8"] else None
        row = 0
        for b, (t, n) in enumerate(zip(total, new)):
            y = wide[x][row:row + n]
            row += n
            pos = torch.arange(t - n, t, device=DEV)
            where = (s["table"][b].long()[pos // c["page"]], pos % c["page"])
            if c["fp8"]:
                scale = y.abs().amax(-1) / 448
                scales[where] = torch.where(scale > 0, scale, 1.0)
                pages[where] = y / scales[where][..., None]
            else:
                pages[where] = y
        res[x + "_pages"] = pages
        if c["fp8"]:
            res[x + "_scale"] = scales
    return res


def _exact_decode(s):
    c = s["case"]
    out, lse = [], []
    r = c["H"] // c["G"]
    for b, n in enumerate(lengths(c)[0]):
        ids = s["table"][b, :-(-n // c["page"])].long()
        kv = []
        for x in ("k", "v"):
            y = s[x + "_pages"][ids]
            y = y.view(torch.float8_e4m3fn).double() * s[x + "_scale"][ids].double()[..., None] if c["fp8"] else y.double()
            kv.append(y.flatten(0, 1)[:n])
        for g in range(c["G"]):
            z = s["q"][b, g * r:(g + 1) * r].double() @ kv[0][:, g].t() / math.sqrt(D)
            lse.append(torch.logsumexp(z, -1))
            out.append(torch.softmax(z, -1) @ kv[1][:, g])
    return {"out": torch.cat(out).view(c["B"], c["H"], D), "lse": torch.cat(lse).view(c["B"], c["H"])}


def _exact_dense(s):
    c = s["case"]
    training = c["op"] == "training"
    r = c["H"] // c["G"]
    wide = {x: s[x].double() for x in ("q", "k", "v")}
    out, lse = torch.zeros_like(wide["q"]), torch.zeros_like(s["lse"], dtype=torch.float64)
    dq, dk, dv = (torch.zeros_like(wide[x]) for x in ("q", "k", "v"))
    q0 = k0 = 0
    for t, n in zip(*lengths(c)):
        for h in range(c["H"]):
            k, v = wide["k"][k0:k0 + t, h // r], wide["v"][k0:k0 + t, h // r]
            for a in range(0, n, 4096):         # a few query rows at a time
                rows = slice(q0 + a, q0 + min(n, a + 4096))
                i = torch.arange(a, min(n, a + 4096), device=DEV)[:, None] + t - n
                q = wide["q"][rows, h]
                z = (q @ k.t()).div_(math.sqrt(D))
                z.masked_fill_(torch.arange(t, device=DEV)[None] > i, -math.inf)
                lse[rows, h] = torch.logsumexp(z, -1)
                p = torch.softmax(z, -1)
                out[rows, h] = p @ v
                if training:
                    do = s["dout"][rows, h].double()
                    dv[k0:k0 + t, h // r] += p.t() @ do
                    dp = do @ v.t()
                    ds = p * (dp - (p * dp).sum(-1, keepdim=True)) / math.sqrt(D)
                    dq[rows, h] = ds @ k
                    dk[k0:k0 + t, h // r] += ds.t() @ q
        q0, k0 = q0 + n, k0 + t
    return {"out": out, "dq": dq, "dk": dk, "dv": dv} if training else {"out": out, "lse": lse}
