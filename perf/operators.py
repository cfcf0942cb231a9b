"""Latent attention (MLA) and its paged cache: what is measured, in plain form and by the library's calls.

Four operators, as a hybrid stack of KDA and latent-attention layers uses them:

* append  -- ``mla_append``: RMSNorm of the latent, position rotation of the shared key part and of the
  queries' part, rows written to a paged cache;
* decode  -- ``mla_decode``: absorbed attention of n tokens per sequence over the paged latent cache;
* prefill -- ``mla_prefill``: expanded causal attention over packed sequences, keys' rotated part shared by heads;
* train   -- ``mla_prefill`` and ``mla_backward``: output and every gradient.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def _ints(text):
    """Lengths as a case holds them: items apart by commas, each "a", "a*n" (a, n times) or "a+s*n" (n numbers from a in steps of s)."""
    out = []
    for item in text.split(","):
        a, _, n = item.partition("*")
        a, _, s = a.partition("+")
        out += [int(a) + int(s or 0) * i for i in range(int(n or 1))]
    return out


def _text(numbers):
    return ",".join(str(n) for n in numbers)


# ---------------------------------------------------------------- cases
def listed():
    return [
        # one serving step of 256 sequences: each appends one token, 32 heads' queries are rotated
        dict(name="append_step_256", op="append", dtype="bf16", lens="1*256", past="16+3*256",
             H=32, dc=512, dr=64, page=64, interleaved=False, packed=False),
        # eight prompts of 8192 tokens enter the cache; the packed rows are kept for the expansion product
        dict(name="append_prompt_8x8192", op="append", dtype="bf16", lens="8192*8", past="0*8", H=32, dc=512,
             dr=64, page=64, interleaved=True, packed=True),
        # the smallest decode: one user, a short context, latency counts
        dict(name="decode_1x1023", op="decode", dtype="bf16", lens="1023", n=1, H=32, dc=512, dr=64, page=64),
        # a full serving batch at uneven contexts, one token each
        dict(name="decode_256x4096", op="decode", dtype="bf16", lens="2048+17*256",
             n=1, H=32, dc=512, dr=64, page=64),
        # four drafted tokens per sequence checked at once, long contexts
        dict(name="decode_tokens_24x16k", op="decode", dtype="bf16", lens="12000+377*24", n=4,
             H=32, dc=512, dr=64, page=32),
        # float32 with odd sizes: small latent, pages of 16, an empty sequence
        dict(name="decode_9x3k_f32", op="decode", dtype="f32", lens="3001,17,0,1500,2999,1,640,2222,2875",
             n=1, H=12, dc=256, dr=32, page=16),
        # a short ragged batch of prompts
        dict(name="prefill_short", op="prefill", dtype="bf16", q_lens="37,201,1,130", past="0*4", H=32,
             dn=128, dr=64, dv=128),
        # two long prompts
        dict(name="prefill_2x8192", op="prefill", dtype="bf16", q_lens="8192*2", past="0*2", H=32, dn=128,
             dr=64, dv=128),
        # the next chunk of prompts whose earlier keys were expanded again from the cache
        dict(name="prefill_chunk_4x1k_on_7k", op="prefill", dtype="bf16", q_lens="1024,777,1000,513",
             past="7000,6500,4097,5555", H=32, dn=128, dr=64, dv=128),
        # a training step's attention, four sequences of 4096
        dict(name="train_4x4096", op="train", dtype="bf16", q_lens="4096*4", past="0*4", H=32, dn=128, dr=64,
             dv=128),
        # packed documents of odd lengths
        dict(name="train_ragged", op="train", dtype="bf16", q_lens="1,777,2049,130,1500,64", past="0*6", H=16,
             dn=128, dr=64, dv=128),
        # float32 training at small odd head sizes
        dict(name="train_f32", op="train", dtype="f32", q_lens="700,33,1025", past="0*3", H=4, dn=72, dr=24,
             dv=80),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "decode", "prefill", "train"])
    bf = rng.random() < 0.75
    dtype = "bf16" if bf else "f32"
    if op == "append":
        n = _log(rng, 1, 256)
        most = max(1, 40000 // n)
        lens = [_log(rng, 1, most) if i == 0 or rng.random() < 0.9 else 0 for i in range(n)]
        dc, dr = rng.choice([(512, 64), (512, 64), (256, 64), (384, 32), (192, 16)])
        return dict(op=op, dtype=dtype, lens=_text(lens), past=_text(rng.randrange(0, 600) for _ in lens),
                    H=rng.choice([1, 4, 7, 16, 32]), dc=dc, dr=dr, page=rng.choice([1, 16, 32, 64, 128]),
                    interleaved=rng.random() < 0.5, packed=rng.random() < 0.5)
    if op == "decode":
        B = _log(rng, 1, 192)
        L = _log(rng, 1, min(65536, (400000 if bf else 60000) // B))
        lens = [max(0, int(L * rng.uniform(0.5, 1.0)) - rng.choice([0, 0, 0, 5])) for _ in range(B)]
        lens[0] = L
        n = rng.choice([1, 1, 2, 3, 4])
        H = rng.choice([1, 8, 12, 16, 32, 32, 64])
        if bf:
            dc, dr = rng.choice([(512, 64), (512, 64), (256, 64), (512, 0), (128, 64)])
        else:
            dc, dr = rng.choice([(512, 64), (256, 32), (100, 20), (64, 0)])
            H = min(H, 16)
        return dict(op=op, dtype=dtype, lens=_text(lens), n=n, H=H, dc=dc, dr=dr, page=rng.choice([16, 32, 64, 128]))
    n = rng.randint(1, 6)
    if bf:
        dn, dr, dv = rng.choice([(128, 64, 128), (128, 64, 128), (128, 64, 128), (128, 0, 128), (64, 32, 64)])
        most, H = (4096 if op == "prefill" else 2500), rng.choice([2, 5, 16, 24])
        if dn == 64:
            most, H = 600, min(H, 5)
    else:
        dn, dr, dv = rng.choice([(128, 64, 128), (72, 24, 80), (33, 7, 65), (64, 0, 64)])
        most, H = 900, rng.choice([1, 3, 8])
    q_lens = [_log(rng, 16 if i == 0 else 1, most) for i in range(n)]
    past = [_log(rng, 1, 2000 if bf else 300) if op == "prefill" and rng.random() < 0.4 else 0 for _ in q_lens]
    return dict(op=op, dtype=dtype, q_lens=_text(q_lens), past=_text(past), H=H, dn=dn, dr=dr, dv=dv)


# ---------------------------------------------------------------- inputs
def _offsets(lens):
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    return cu


def _pages(lens, page, gen):
    """A page table whose pages lie in a random order in the pool, as a running server's do."""
    need = [-(-n // page) for n in lens]
    total, width = sum(need), max(max(need), 1)
    order = torch.randperm(total, generator=gen, device="cuda").to(torch.int32)
    table = torch.zeros(len(lens), width, dtype=torch.int32, device="cuda")
    cols = torch.arange(width, device="cuda")
    table[cols[None, :] < torch.tensor(need, device="cuda")[:, None]] = order
    return table, max(total, 1)


def _inv_freq(dr):
    return 10000.0 ** (-torch.arange(0, dr, 2, dtype=torch.float64) / dr)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    dt = DTYPES[case["dtype"]]
    rand = lambda *s: torch.randn(*s, generator=gen, device="cuda", dtype=torch.float32).to(dt)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    st = dict(case=case)
    if case["op"] == "append":
        lens, past, dc, dr = _ints(case["lens"]), _ints(case["past"]), case["dc"], case["dr"]
        cu, T = _offsets(lens), sum(lens)
        ends = [p + n for p, n in zip(past, lens)]
        st["page_table"], pages = _pages(ends, case["page"], gen)
        st["cache"] = rand(pages, case["page"], dc + dr)
        proj = 1.5 * rand(T, dc + dr)               # one projection holds the latent and the shared key part
        st["c"], st["k_rope"] = proj[:, :dc], proj[:, dc:]
        st["q"] = rand(T, case["H"], 128 + dr)      # the queries' projection: unrotated part first
        st["past"], st["cu"] = i32(past), i32(cu)
        st["norm_weight"] = 1.0 + 0.1 * torch.randn(dc, generator=gen, device="cuda")
        st["inv_freq"] = _inv_freq(dr).to("cuda", torch.float32)
        st["q_out"] = torch.empty(T, case["H"], dr, dtype=dt, device="cuda")
        return st
    if case["op"] == "decode":
        lens = _ints(case["lens"])
        B, W = len(lens), case["dc"] + case["dr"]
        st["page_table"], pages = _pages(lens, case["page"], gen)
        st["cache"] = rand(pages, case["page"], W)
        st["q"] = rand(B, case["n"], case["H"], W)
        st["lens"] = i32(lens)
        st["longest"] = max(lens)
        st["scale"] = 1.0 / math.sqrt(128 + case["dr"])
        return st
    H, dn, dr, dv = case["H"], case["dn"], case["dr"], case["dv"]
    ql = _ints(case["q_lens"])
    kl = [a + b for a, b in zip(ql, _ints(case["past"]))]
    cq, ck = _offsets(ql), _offsets(kl)
    st["longest_q"], st["longest_k"] = max(ql), max(kl)
    st["q"] = rand(cq[-1], H, dn + dr)
    kv = rand(ck[-1], H, dn + dv)                   # the expansion product's output: keys and values side by side
    st["k"], st["v"] = kv[..., :dn], kv[..., dn:]
    st["k_rope"] = rand(ck[-1], dr) if dr else None
    st["cu_q"], st["cu_k"] = i32(cq), i32(ck)
    st["cu_q_host"], st["cu_k_host"] = (torch.tensor(c, dtype=torch.int32) for c in (cq, ck))
    if case["op"] == "train":
        st["dO"] = rand(cq[-1], H, dv)
    return st


# ---------------------------------------------------------------- one pass
def run(st):
    if own:
        return _own(st)
    return {"append": _plain_append, "decode": _plain_decode, "prefill": _plain_prefill,
            "train": _plain_train}[st["case"]["op"]](st)


def _own(st):
    import gated_delta_rule_126_b200 as lib
    case = st["case"]
    if case["op"] == "append":
        out = lib.mla_append(st["c"], st["k_rope"], st["cache"], st["page_table"], st["past"], st["cu"],
                             norm_weight=st["norm_weight"], eps=1e-6, inv_freq=st["inv_freq"],
                             interleaved=case["interleaved"], q_rope=st["q"][..., 128:], packed=case["packed"],
                             out={"q_rope": st["q_out"]})
        res = dict(cache=st["cache"], q_rope=out["q_rope"])
        if case["packed"]:
            res.update(c=out["c"], k_rope=out["k_rope"])
        return res
    if case["op"] == "decode":
        return lib.mla_decode(st["q"], st["cache"], st["page_table"], st["lens"], d_latent=case["dc"],
                              scale=st["scale"])[0]
    args = (st["q"], st["k"], st["v"], st["cu_q"], st["cu_k"])
    host = dict(k_rope=st["k_rope"], cu_q_host=st["cu_q_host"], cu_k_host=st["cu_k_host"], causal=True)
    if case["op"] == "prefill":
        return lib.mla_prefill(*args, **host)[0]
    o, lse = lib.mla_prefill(*args, **host, want_lse=True)
    g = lib.mla_backward(*args, o, lse, st["dO"], **host)
    return dict(o=o, **{n: g[n] for n in ("dq", "dk", "dv")}, **({"dk_rope": g["dk_rope"]} if case["dr"] else {}))


def _rotate(x, ang, interleaved):
    """x [T, ..., dr] turned by ang [T, dr/2] (float64 angles, float32 products)."""
    shape = (ang.shape[0],) + (1,) * (x.dim() - 2) + (ang.shape[1],)
    cos, sin = ang.cos().float().view(shape), ang.sin().float().view(shape)
    if interleaved:
        a, b = x[..., 0::2], x[..., 1::2]
        return torch.stack((a * cos - b * sin, a * sin + b * cos), -1).flatten(-2)
    a, b = x.chunk(2, -1)
    return torch.cat((a * cos - b * sin, a * sin + b * cos), -1)


def _plain_append(st):
    case, dt = st["case"], st["c"].dtype
    T = st["c"].shape[0]
    lens = (st["cu"][1:] - st["cu"][:-1]).long()
    b = torch.repeat_interleave(torch.arange(lens.shape[0], device="cuda"), lens, output_size=T)
    pos = torch.arange(T, device="cuda") - st["cu"].long()[b] + st["past"].long()[b]
    c = st["c"].float()
    c = c / torch.sqrt((c * c).mean(-1, keepdim=True) + 1e-6) * st["norm_weight"]
    ang = pos.double()[:, None] * st["inv_freq"].double()
    k = _rotate(st["k_rope"].float(), ang, case["interleaved"])
    q = _rotate(st["q"][..., 128:].float(), ang, case["interleaved"])
    c, k = c.to(dt), k.to(dt)
    P = case["page"]
    slot = st["page_table"].long()[b, pos // P] * P + pos % P
    st["cache"].view(-1, case["dc"] + case["dr"])[slot] = torch.cat((c, k), -1)
    st["q_out"].copy_(q)
    res = dict(cache=st["cache"], q_rope=st["q_out"])
    if case["packed"]:
        res.update(c=c, k_rope=k)
    return res


def _softmax(s, seen):
    """Rows of s over the seen places; a row that sees nothing is all zeros. Works in place on s."""
    s.masked_fill_(~seen, -math.inf)
    m = s.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    s.sub_(m).exp_()
    z = s.sum(-1, keepdim=True)
    return s.div_(torch.where(z == 0, torch.ones_like(z), z))


def _plain_decode(st):
    case = st["case"]
    B, n, H, W = st["q"].shape
    dc = case["dc"]
    L = max(st["longest"], 1)
    pos = torch.arange(L, device="cuda")
    P = case["page"]
    slot = st["page_table"].long()[:, pos // P] * P + pos % P
    rows = st["cache"].view(-1, W)[slot].float()                              # [B, L, W]
    q = st["q"].float().view(B, n * H, W)
    s = torch.bmm(q, rows.transpose(1, 2)).view(B, n, H, L).mul_(st["scale"])
    end = st["lens"].long()[:, None] - (n - 1) + torch.arange(n, device="cuda")  # [B, n]
    p = _softmax(s, (pos < end[..., None])[:, :, None, :])
    return torch.bmm(p.view(B, n * H, L), rows[..., :dc]).view(B, n, H, dc).to(st["q"].dtype)


def _padded(cu, width):
    """[N, width] row numbers (clamped to the tensor) and which of them are a sequence's own."""
    cu = cu.long()
    at = torch.arange(width, device="cuda")
    own_rows = at < (cu[1:] - cu[:-1])[:, None]
    return torch.where(own_rows, cu[:-1, None] + at, 0), own_rows


def _plain_scores(st):
    case = st["case"]
    Lq, Lk = st["longest_q"], st["longest_k"]
    qi, qm = _padded(st["cu_q"], Lq)
    ki, km = _padded(st["cu_k"], Lk)
    q = st["q"].float()[qi].transpose(1, 2)                                    # [N, H, Lq, d]
    k = st["k"].float()
    if case["dr"]:
        k = torch.cat((k, st["k_rope"].float()[:, None].expand(-1, case["H"], -1)), -1)
    k = k[ki].transpose(1, 2)
    v = st["v"].float()[ki].transpose(1, 2)
    lq, lk = qm.sum(1), km.sum(1)
    seen = torch.arange(Lk, device="cuda") <= (torch.arange(Lq, device="cuda") + (lk - lq)[:, None])[..., None]
    seen = (seen & km[:, None, :] & qm[:, :, None])[:, None]
    scale = 1.0 / math.sqrt(case["dn"] + case["dr"])
    p = _softmax(torch.matmul(q, k.transpose(2, 3)).mul_(scale), seen)
    return q, k, v, p, qi, qm, ki, km, scale


def _plain_prefill(st):
    _, _, v, p, _, qm, _, _, _ = _plain_scores(st)
    return torch.matmul(p, v).transpose(1, 2)[qm].to(st["q"].dtype)


def _plain_train(st):
    case, dt = st["case"], st["q"].dtype
    q, k, v, p, qi, qm, ki, km, scale = _plain_scores(st)
    o = torch.matmul(p, v)
    dO = (st["dO"].float()[qi] * qm[..., None, None]).transpose(1, 2)
    dv = torch.matmul(p.transpose(2, 3), dO)
    ds = torch.matmul(dO, v.transpose(2, 3)).sub_((dO * o).sum(-1, keepdim=True)).mul_(p).mul_(scale)
    dq = torch.matmul(ds, k)
    dk = torch.matmul(ds.transpose(2, 3), q)
    rows = lambda x, m: x.transpose(1, 2)[m]
    dk = rows(dk, km)
    res = dict(o=rows(o, qm).to(dt), dq=rows(dq, qm).to(dt), dk=dk[..., :case["dn"]].to(dt), dv=rows(dv, km).to(dt))
    if case["dr"]:
        res["dk_rope"] = dk[..., case["dn"]:].sum(1).to(dt)
    return res


# ---------------------------------------------------------------- what a pass cannot do without
def _pairs(case):
    """(query, key) pairs that the causal mask leaves."""
    return sum(n * p + n * (n + 1) // 2 for n, p in zip(_ints(case["q_lens"]), _ints(case["past"])))


def work(case):
    es = 2 if case["dtype"] == "bf16" else 4
    H, dr = case["H"], case["dr"]
    if case["op"] == "append":
        T, W = sum(_ints(case["lens"])), case["dc"] + dr
        return dict(bytes=T * es * (W * (3 if case["packed"] else 2) + 2 * H * dr), flops=T * (4 * case["dc"] + 3 * dr * (H + 1)))
    if case["op"] == "decode":
        W, dc, n, lens = case["dc"] + dr, case["dc"], case["n"], _ints(case["lens"])
        seen = sum(max(0, L - (n - 1) + i) for L in lens for i in range(n))
        return dict(bytes=es * (sum(lens) * W + len(lens) * n * H * (W + dc)),
                    flops=2 * seen * H * (W + dc))
    d, dv, dn = case["dn"] + dr, case["dv"], case["dn"]
    Tq = sum(_ints(case["q_lens"]))
    Tk = Tq + sum(_ints(case["past"]))
    read = Tq * H * d + Tk * (H * (dn + dv) + dr)
    if case["op"] == "prefill":
        return dict(bytes=es * (read + Tq * H * dv), flops=2 * _pairs(case) * H * (d + dv))
    # forward, then dO V^T, P^T dO, dS K and dS^T Q; the scores' recomputation is not counted
    return dict(bytes=es * (2 * read + 2 * Tq * H * dv), flops=2 * _pairs(case) * H * (3 * d + 3 * dv))


# ---------------------------------------------------------------- 64 bits, one sequence and head at a time
def exact(case, seed):
    st = prepare(case, seed)
    f = lambda t: t.double()
    if case["op"] == "append":
        cache, T, P = f(st["cache"]), st["c"].shape[0], case["page"]
        pos = torch.cat([torch.arange(p, p + n) for p, n in zip(_ints(case["past"]), _ints(case["lens"]))])
        c = f(st["c"])
        c = c * (c.square().mean(1) + 1e-6).rsqrt()[:, None] * f(st["norm_weight"])
        turn = torch.polar(torch.ones(T, case["dr"] // 2, dtype=torch.float64, device="cuda"),
                           pos.cuda().double()[:, None] * f(st["inv_freq"]))

        def turned(x, t):
            if case["interleaved"]:
                return torch.view_as_real(torch.view_as_complex(f(x).unflatten(-1, (-1, 2)).contiguous()) * t).flatten(-2)
            h = case["dr"] // 2
            z = torch.complex(f(x)[..., :h].contiguous(), f(x)[..., h:].contiguous()) * t
            return torch.cat((z.real, z.imag), -1)

        k = turned(st["k_rope"], turn)
        at, table = 0, st["page_table"].cpu()
        for b, (p, n) in enumerate(zip(_ints(case["past"]), _ints(case["lens"]))):
            where = torch.arange(p, p + n)
            page = table[b][torch.div(where, P, rounding_mode="floor")].long()
            cache[page.cuda(), (where % P).cuda()] = torch.cat((c, k), 1)[at:at + n]
            at += n
        res = dict(cache=cache, q_rope=turned(st["q"][..., 128:], turn[:, None]))
        if case["packed"]:
            res.update(c=c, k_rope=k)
        return res
    if case["op"] == "decode":
        B, n, H, W = st["q"].shape
        o = torch.zeros(B, n, H, case["dc"], dtype=torch.float64, device="cuda")
        for b, L in enumerate(_ints(case["lens"])):
            rows = f(st["cache"][st["page_table"][b].long()]).reshape(-1, W)[:L]
            for i in range(n):
                end = L - (n - 1) + i
                if end > 0:
                    s = f(st["q"][b, i]) @ rows[:end].T * st["scale"]
                    o[b, i] = torch.softmax(s, 1) @ rows[:end, :case["dc"]]
        return o
    H, dn, dr = case["H"], case["dn"], case["dr"]
    scale = (dn + dr) ** -0.5
    cq, ck = st["cu_q_host"].tolist(), st["cu_k_host"].tolist()
    z = lambda t: torch.zeros(t.shape, dtype=torch.float64, device="cuda")
    o = torch.zeros(cq[-1], H, case["dv"], dtype=torch.float64, device="cuda")
    g = dict(dq=z(st["q"]), dk=z(st["k"]), dv=z(st["v"]), **({"dk_rope": z(st["k_rope"])} if dr else {}))
    for b, (n, past) in enumerate(zip(_ints(case["q_lens"]), _ints(case["past"]))):
        qs, ks = slice(cq[b], cq[b + 1]), slice(ck[b], ck[b + 1])
        hidden = torch.ones(n, n + past, dtype=torch.bool, device="cuda").triu(past + 1)
        for h in range(H):
            q, k, v = f(st["q"][qs, h]), f(st["k"][ks, h]), f(st["v"][ks, h])
            if dr:
                k = torch.cat((k, f(st["k_rope"][ks])), 1)
            p = torch.softmax((q @ k.T * scale).masked_fill(hidden, -math.inf), 1)
            o[qs, h] = p @ v
            if case["op"] == "train":
                dO = f(st["dO"][qs, h])
                dp = dO @ v.T
                ds = p * (dp - (p * dp).sum(1, keepdim=True)) * scale
                g["dv"][ks, h] = p.T @ dO
                g["dq"][qs, h] = ds @ k
                dk = ds.T @ q
                g["dk"][ks, h] = dk[:, :dn]
                if dr:
                    g["dk_rope"][ks] += dk[:, dn:]
    return o if case["op"] == "prefill" else dict(o=o, **g)
