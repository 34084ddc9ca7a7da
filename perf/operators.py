"""The attention half of a decoder layer between the q/k/v linears and o_proj:
rotary positions with the append to a paged key/value cache, causal attention
over packed prompts, and decode attention for a batch with a shared prefix.

`run` computes them in plain torch operations (32-bit arithmetic, rounded to
bf16 once) or, when `own` is set, through the package's entry points.
"""
import math
import random

import numpy as np
import torch

own = False

BF = torch.bfloat16


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------
def _text(lens):
    return ",".join(str(int(n)) for n in lens)


def _lens(text):
    return [int(n) for n in text.split(",")]


def _rope(name, q_lens, past, hq, hkv, d, page, rot, layout="half", norm=False, theta=10000.0, scaling="none",
          factor=1.0):
    return dict(name=name, op="rope_append", q_lens=_text(q_lens), past=_text(past), hq=hq, hkv=hkv, d=d, page=page,
                rot=rot, layout=layout, norm=norm, theta=theta, scaling=scaling, factor=factor)


def _prefill(name, q_lens, past, hq, hkv, d, page):
    return dict(name=name, op="attn_prefill", q_lens=_text(q_lens), past=_text(past), hq=hq, hkv=hkv, d=d, page=page)


def _decode(name, kv_lens, prefix, hq, hkv, d, page):
    return dict(name=name, op="attn_decode", kv_lens=_text(kv_lens), prefix=prefix, hq=hq, hkv=hkv, d=d, page=page)


def _spread(n, lo, hi, seed):
    """n lengths in [lo, hi], the same ones for the same arguments."""
    r = random.Random(seed)
    return [r.randint(lo, hi) for _ in range(n)]


def listed():
    return [
        # one decode step of 16 sequences, 7B heads (as many key heads as query heads): latency
        _rope("rope_decode16", [1] * 16, _spread(16, 1500, 4000, 1), 32, 32, 128, 64, 128),
        # a 2048-token prompt, 7B heads: the prefill step's shape
        _rope("rope_prompt2048", [2048], [0], 32, 32, 128, 64, 128),
        # packed ragged prompts and chunks far into long contexts, grouped heads with norms, half of each head
        # rotated in neighbouring pairs, frequencies scaled by parts
        _rope("rope_packed_norm", [1, 333, 1024, 129, 2049, 64, 4000], [120000, 0, 7001, 31, 0, 65535, 500], 32, 8,
              128, 16, 64, layout="interleaved", norm=True, theta=500000.0, scaling="by_parts", factor=8.0),
        # a short question, one sequence: latency of a first token
        _prefill("prefill_short33", [33], [0], 32, 8, 128, 64),
        # the 7B prefill step: one 2048-token prompt, 32 heads each with its own keys
        _prefill("prefill_prompt2048", [2048], [0], 32, 32, 128, 64),
        # packed prompts of very different lengths, grouped heads (8B), small pages
        _prefill("prefill_packed_gqa", [1, 127, 128, 129, 700, 1500, 1511], [0] * 7, 32, 8, 128, 16),
        # chunked prompts: 512 and 257 new tokens over 7 and 3 thousand cached ones, heads of 64
        _prefill("prefill_chunks_d64", [512, 257], [7167, 3201], 32, 8, 64, 128),
        # a long document
        _prefill("prefill_long16k", [16384], [0], 32, 8, 128, 64),
        # one user, one long context, grouped heads: latency and the split of one sequence over the GPU
        _decode("decode_one_8k", [8191], 0, 32, 8, 128, 64),
        # 16 users with ragged contexts, 7B heads (the decode step's M = 16)
        _decode("decode16_ragged", _spread(16, 700, 4090, 2), 0, 32, 32, 128, 64),
        # 64 users that share an 8192-token system prompt, each with its own short continuation
        _decode("decode64_prefix8k", [8192 + n for n in _spread(64, 1, 511, 3)], 8192, 32, 8, 128, 64),
        # 16 users with long contexts, grouped heads
        _decode("decode16_32k", _spread(16, 20000, 32768, 4), 0, 32, 8, 128, 64),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope_append", "attn_prefill", "attn_decode"])
    hkv, g = rng.choice([(32, 1), (8, 4), (4, 8), (2, 7), (12, 1), (1, 16), (5, 3)])
    d = rng.choice([64, 128, 128])
    page = rng.choice([16, 32, 64, 128, 256])
    hq = hkv * g
    if op == "rope_append":
        n = _log(rng, 1, 32)
        total = _log(rng, n, 8192)
        q = [max(1, total // n + rng.randint(-(total // (2 * n)), total // (2 * n))) for _ in range(n)]
        past = [rng.choice([0, rng.randint(0, 200), _log(rng, 200, 120000)]) for _ in range(n)]
        rot = rng.choice([d, d, d // 2, d // 4])
        scaling = rng.choice(["none", "linear", "by_parts"])
        c = _rope("", q, past, hq, hkv, d, page, rot, rng.choice(["half", "interleaved"]), rng.random() < 0.5,
                  rng.choice([10000.0, 500000.0]), scaling, 1.0 if scaling == "none" else rng.choice([4.0, 8.0]))
    elif op == "attn_prefill":
        n = _log(rng, 1, 16)
        total = _log(rng, n, 8192)
        q = [max(1, total // n + rng.randint(-(total // (2 * n)), total // (2 * n))) for _ in range(n)]
        past = [rng.choice([0, 0, rng.randint(0, 300), _log(rng, 300, 8000)]) for _ in range(n)]
        c = _prefill("", q, past, hq, hkv, d, page)
    else:
        n = _log(rng, 1, 64)
        prefix = rng.choice([0, 0, max(1, _log(rng, 256, 16384) // page) * page])
        hi = _log(rng, 16, max(64, min(65536, 3200000 // (n * hkv))))
        kv = [prefix + rng.randint(1, hi) for _ in range(n)]
        c = _decode("", kv, prefix, hq, hkv, d, page)
    del c["name"]
    return c


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------
def _rows(gen, n, heads, d, outliers):
    """n rows of heads, as a linear writes them; a few channels of a head are
    larger than the rest when `outliers` (keys and queries)."""
    x = torch.randn((n, heads, d), generator=gen, device="cuda", dtype=torch.float32)
    if outliers:
        big = torch.rand((1, heads, d), generator=gen, device="cuda") < 0.03
        x = torch.where(big, 3.0 * x, x)
    return x.to(BF).reshape(n, heads * d)


def _table(gen, counts, shared, n_pages):
    """Page table of sequences with `counts` pages each, the first `shared`
    of them common to all, out of pages in random order; entries past a
    sequence's end are -1."""
    perm = torch.randperm(n_pages, generator=gen, device="cuda").to(torch.int32).cpu().numpy()
    t = np.full((len(counts), max(1, max(counts))), -1, np.int32)
    at = shared
    for b, c in enumerate(counts):
        t[b, :min(c, shared)] = perm[:min(c, shared)]
        own_pages = max(0, c - shared)
        t[b, shared:shared + own_pages] = perm[at:at + own_pages]
        at += own_pages
    return torch.from_numpy(t).cuda()


def _inputs(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed * 1000003 + 17)
    hq, hkv, d, page = case["hq"], case["hkv"], case["d"], case["page"]
    s = dict(case=case)
    if case["op"] == "attn_decode":
        kv = _lens(case["kv_lens"])
        q_lens = [1] * len(kv)
        prefix = case["prefix"]
    else:
        q_lens = _lens(case["q_lens"])
        kv = [n + p for n, p in zip(q_lens, _lens(case["past"]))]
        prefix = 0
    s["host"] = (q_lens, kv)
    T = sum(q_lens)
    s["cu_q"] = torch.tensor([0] + list(np.cumsum(q_lens)), dtype=torch.int32, device="cuda")
    s["kv_len"] = torch.tensor(kv, dtype=torch.int32, device="cuda")
    counts = [-(-n // page) for n in kv]
    if case["op"] == "rope_append":
        # only the pages that the new tokens fall into exist: the rest of a long context does not matter here
        first = [(n - m) // page for n, m in zip(kv, q_lens)]
        n_pages = sum(c - f for c, f in zip(counts, first)) + 1
        t = np.full((len(kv), max(counts)), -1, np.int32)
        perm = torch.randperm(n_pages, generator=gen, device="cuda").to(torch.int32).cpu().numpy()
        at = 0
        for b, (c, f) in enumerate(zip(counts, first)):
            t[b, f:c] = perm[at:at + c - f]
            at += c - f
        s["table"] = torch.from_numpy(t).cuda()
        qkv = [_rows(gen, T, h, d, o) for h, o in ((hq, True), (hkv, True), (hkv, False))]
        s["q"], s["k"], s["v"] = qkv
        if case["norm"]:
            s["qw"] = (1.0 + 0.2 * torch.randn(d, generator=gen, device="cuda")).to(BF)
            s["kw"] = (1.0 + 0.2 * torch.randn(d, generator=gen, device="cuda")).to(BF)
        s["kc"] = torch.zeros((n_pages, hkv, page, d), dtype=BF, device="cuda")
        s["vc"] = torch.zeros((n_pages, hkv, page, d), dtype=BF, device="cuda")
    else:
        shared = prefix // page
        n_pages = shared + sum(c - shared for c in counts) + 1
        s["table"] = _table(gen, counts, shared, n_pages)
        s["q"] = _rows(gen, T, hq, d, True)
        s["kc"] = _rows(gen, n_pages * page, hkv, d, True).view(n_pages, page, hkv, d).transpose(1, 2).contiguous()
        s["vc"] = _rows(gen, n_pages * page, hkv, d, False).view(n_pages, page, hkv, d).transpose(1, 2).contiguous()
    return s


LOW, HIGH, ORIGINAL = 1.0, 4.0, 8192.0  # of the frequencies scaled by parts


def prepare(case, seed):
    s = _inputs(case, seed)
    if own:
        from w4a4_rank_gemm_b200 import serq as S
        s["cache"] = S.KVCache(K=s["kc"], V=s["vc"])
        s["out"] = torch.empty_like(s["q"])
        if case["op"] == "rope_append":
            s["rope"] = S.Rope(case["d"], rot_dim=case["rot"], layout=case["layout"], theta=case["theta"],
                               scaling=case["scaling"], factor=case["factor"], original_len=ORIGINAL, low=LOW,
                               high=HIGH)
        elif case["op"] == "attn_prefill":
            s["ws"] = S.attn_prefill_ws(s["cache"], s["q"].shape[0], case["hq"], s["kv_len"].shape[0],
                                        s["table"].shape[1])
        else:
            s["ws"] = S.attn_decode_ws(s["cache"], s["q"].shape[0], case["hq"], s["table"].shape[1], case["prefix"])
    return s


# --------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------
def run(state):
    op = state["case"]["op"]
    if own:
        from w4a4_rank_gemm_b200 import serq as S
        if op == "rope_append":
            S.rope_append(state["rope"], state["cache"], state["q"], state["k"], state["v"], state["cu_q"],
                          state["kv_len"], state["table"], q_weight=state.get("qw"), k_weight=state.get("kw"),
                          eps=1e-6, Qout=state["out"])
            return state["out"], state["kc"], state["vc"]
        if op == "attn_prefill":
            return S.attn_prefill(state["cache"], state["q"], state["cu_q"], state["kv_len"], state["table"],
                                  O=state["out"], ws=state["ws"])
        return S.attn_decode(state["cache"], state["q"], state["kv_len"], state["table"],
                             prefix_len=state["case"]["prefix"], O=state["out"], ws=state["ws"])
    if op == "rope_append":
        return _plain_rope_append(state)
    return _plain_attention(state)


def _plain_rope_append(s):
    c = s["case"]
    d, page, rot, hkv = c["d"], c["page"], c["rot"], c["hkv"]
    cu, kv = s["cu_q"].long(), s["kv_len"].long()
    T = s["q"].shape[0]
    t = torch.arange(T, device="cuda")
    b = torch.searchsorted(cu, t, right=True) - 1
    pos = kv[b] - (cu[b + 1] - t)
    # angles in 64 bits: a far position times a frequency loses its fraction in 32
    i = torch.arange(rot // 2, device="cuda", dtype=torch.float64)
    f = torch.exp(-math.log(c["theta"]) * 2.0 * i / rot)
    if c["scaling"] == "linear":
        f = f / c["factor"]
    elif c["scaling"] == "by_parts":
        r = ORIGINAL * f / (2.0 * math.pi)
        keep = torch.clamp((r - LOW) / (HIGH - LOW), 0.0, 1.0)
        f = (1.0 - keep) * f / c["factor"] + keep * f
    ang = pos.double()[:, None] * f[None, :]
    cos, sin = torch.cos(ang).float()[:, None, :], torch.sin(ang).float()[:, None, :]

    def turn(x, heads, w):
        x = x.view(T, heads, d).float()
        if w is not None:
            x = x / torch.sqrt(torch.sum(x * x, dim=-1, keepdim=True) / d + 1e-6) * w.float()
        y = x.clone()
        if c["layout"] == "half":
            x1, x2 = x[..., :rot // 2], x[..., rot // 2:rot]
            y[..., :rot // 2] = x1 * cos - x2 * sin
            y[..., rot // 2:rot] = x1 * sin + x2 * cos
        else:
            x1, x2 = x[..., 0:rot:2], x[..., 1:rot:2]
            y[..., 0:rot:2] = x1 * cos - x2 * sin
            y[..., 1:rot:2] = x1 * sin + x2 * cos
        return y.to(BF)

    q = turn(s["q"], c["hq"], s.get("qw")).view(T, -1)
    k = turn(s["k"], hkv, s.get("kw"))
    pages = s["table"][b, pos // page].long()
    s["kc"][pages, :, pos % page] = k
    s["vc"][pages, :, pos % page] = s["v"].view(T, hkv, d)
    return q, s["kc"], s["vc"]


def _plain_attention(s):
    c = s["case"]
    hq, hkv, d, page = c["hq"], c["hkv"], c["d"], c["page"]
    g = hq // hkv
    q_lens, kv_lens = s["host"]
    out = torch.empty_like(s["q"])
    at = 0
    for b, (n, kv) in enumerate(zip(q_lens, kv_lens)):
        pages = s["table"][b, :-(-kv // page)].long()
        k = s["kc"][pages].transpose(0, 1).reshape(hkv, -1, d)[:, :kv].float()
        v = s["vc"][pages].transpose(0, 1).reshape(hkv, -1, d)[:, :kv].float()
        step = max(1, (1 << 28) // (hq * kv))
        for r0 in range(0, n, step):
            r1 = min(n, r0 + step)
            q = s["q"][at + r0:at + r1].view(r1 - r0, hkv, g, d).permute(1, 2, 0, 3).reshape(hkv, -1, d).float()
            x = torch.matmul(q, k.transpose(1, 2)).view(hkv, g, r1 - r0, kv) * (1.0 / math.sqrt(d))
            if n > 1:
                pos = kv - n + torch.arange(r0, r1, device="cuda")
                x = torch.where(torch.arange(kv, device="cuda")[None, :] <= pos[:, None], x, float("-inf"))
            p = torch.exp(x - torch.amax(x, dim=-1, keepdim=True))
            z = torch.sum(p, dim=-1, keepdim=True)
            o = torch.matmul(p.view(hkv, -1, kv), v).view(hkv, g, r1 - r0, d) / z
            out[at + r0:at + r1] = o.permute(2, 0, 1, 3).reshape(r1 - r0, hq * d).to(BF)
        at += n
    return out


# --------------------------------------------------------------------------
# what a pass cannot do without, and its values in 64 bits
# --------------------------------------------------------------------------
def work(case):
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    if case["op"] == "rope_append":
        T = sum(_lens(case["q_lens"]))
        per = (hq + 2 * hkv) * d
        # per rotated pair 4 products and 2 sums; a norm adds 4 per element
        return {"bytes": 2.0 * 2 * T * per, "flops": T * (hq + hkv) * (3.0 * case["rot"] + (4.0 * d if case["norm"] else 0))}
    if case["op"] == "attn_prefill":
        q = _lens(case["q_lens"])
        kv = [n + p for n, p in zip(q, _lens(case["past"]))]
        pairs = sum(n * m - n * (n - 1) // 2 for n, m in zip(q, kv))
        return {"bytes": 4.0 * sum(q) * hq * d + 4.0 * sum(kv) * hkv * d, "flops": 4.0 * pairs * hq * d}
    kv, prefix = _lens(case["kv_lens"]), case["prefix"]
    read = prefix + sum(n - prefix for n in kv)
    return {"bytes": 4.0 * len(kv) * hq * d + 4.0 * read * hkv * d, "flops": 4.0 * sum(kv) * hq * d}


def exact(case, seed):
    s = _inputs(case, seed)
    if case["op"] == "rope_append":
        return _exact_rope_append(case, s)
    return _exact_attention(case, s)


def _exact_rope_append(c, s):
    """Rotation as a product of complex numbers, sequence by sequence."""
    d, page, rot = c["d"], c["page"], c["rot"]
    base = c["theta"] ** (-1.0 / (rot // 2))
    f = np.array([base ** j for j in range(rot // 2)], np.float64)
    if c["scaling"] == "linear":
        f /= c["factor"]
    elif c["scaling"] == "by_parts":
        for j in range(rot // 2):
            turns = f[j] * ORIGINAL / (2 * np.pi)
            w = min(max((turns - LOW) / (HIGH - LOW), 0.0), 1.0)
            f[j] = f[j] * (w + (1.0 - w) / c["factor"])
    freq = torch.from_numpy(f).cuda()

    def rotated(x, n, heads, w, first):
        x = x.double().reshape(n, heads, d)
        if w is not None:
            x = x * w.double() * (x.pow(2).mean(-1, keepdim=True) + 1e-6).rsqrt()
        ang = torch.arange(first, first + n, device="cuda", dtype=torch.float64).outer(freq)
        unit = torch.polar(torch.ones_like(ang), ang)[:, None]
        part = x[..., :rot]
        if c["layout"] == "half":
            z = torch.complex(part[..., :rot // 2].contiguous(), part[..., rot // 2:].contiguous()) * unit
            part = torch.cat([z.real, z.imag], -1)
        else:
            z = torch.view_as_complex(part.reshape(n, heads, rot // 2, 2).contiguous()) * unit
            part = torch.view_as_real(z).reshape(n, heads, rot)
        return torch.cat([part, x[..., rot:]], -1)

    kc, vc = s["kc"].double(), s["vc"].double()
    qs, at = [], 0
    for b, (n, kv) in enumerate(zip(*s["host"])):
        rows = slice(at, at + n)
        qs.append(rotated(s["q"][rows], n, c["hq"], s.get("qw"), kv - n).reshape(n, -1))
        k = rotated(s["k"][rows], n, c["hkv"], s.get("kw"), kv - n)
        p = torch.arange(kv - n, kv, device="cuda")
        where = s["table"][b].long()[torch.div(p, page, rounding_mode="floor")]
        kc[where, :, p % page] = k
        vc[where, :, p % page] = s["v"][rows].double().reshape(n, c["hkv"], d)
        at += n
    return torch.cat(qs), kc, vc


def _exact_attention(c, s):
    hq, hkv, d, page = c["hq"], c["hkv"], c["d"], c["page"]
    out = torch.empty((s["q"].shape[0], hq, d), dtype=torch.float64, device="cuda")
    at = 0
    for b, (n, kv) in enumerate(zip(*s["host"])):
        where = s["table"][b, :(kv + page - 1) // page].long()
        rows = max(1, (1 << 26) // kv)
        for h in range(hq):
            k = s["kc"][where, h // (hq // hkv)].reshape(-1, d)[:kv].double()
            v = s["vc"][where, h // (hq // hkv)].reshape(-1, d)[:kv].double()
            for r in range(0, n, rows):
                m = min(rows, n - r)
                # the rows of this block see no key past its last row's position
                see = kv - n + r + m
                logit = s["q"][at + r:at + r + m].view(m, hq, d)[:, h].double() @ k[:see].t() / math.sqrt(d)
                hidden = torch.ones((m, see), dtype=torch.bool, device="cuda").triu(see - m + 1)
                w = torch.softmax(logit.masked_fill(hidden, float("-inf")), dim=-1)
                out[at + r:at + r + m, h] = w @ v[:see]
        at += n
    return out.reshape(-1, hq * d)
