"""The serving operators around a block's compressed matrices, as measured work.

Four operators, each in a plain form (elementary torch operations) and as the
calls a program makes of entropy_decoding_b200.df11:

  extend   df11_kv_extend: pages, block tables, slots, positions and sequence
           starts of one step, from the requests' lengths
  rope     df11_qk_norm_rope: RMS norm of every query and key head and the
           rotation by the token's position, in one pass
  cache    df11_kv4_append, then df11_kv4_gather: keys and values into the
           paged 4-bit cache, and back out as the values it holds
  attend   df11_kv4_attention: queries against the paged 4-bit cache

The 4-bit cache.  Blocks of 16 consecutive elements of a head share a scale s
in FP8 E4M3; an element is one of +-{0, 0.5, 1, 1.5, 2, 3, 4, 6} (E2M1: sign,
two exponent bits, one mantissa bit) and stands for level * s * g, g the
cache's FP32 scale of keys or of values.  For BF16 inputs x (FP32 inputs are
rounded to BF16 first): s = E4M3(min((max |x| / 6) / g, 448)), level =
E2M1(x / (s * g)), both to nearest, ties to even.  One page of one head is a
contiguous block of page_size * head_dim * 9 / 8 bytes: K codes, a row of
head_dim / 2 bytes per token (element 2i in the low nibble of byte i); K
scales, head_dim / 16 bytes per token; V codes, for every 4 tokens and 16
elements the 4 tokens' 8 bytes; V scales, page_size bytes per 16 elements.
"""
import math
import random

import torch

own = False

LEVELS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one decode step of a full batch: a token for each of 128 requests
        dict(name="extend_step", op="extend", reqs=128, kv_min=1, kv_max=8192, new_min=1, new_max=1, page=16,
             pad=0, lens=11),
        # a step that takes in many prompts at once, padded to a fixed token count
        dict(name="extend_prompts", op="extend", reqs=509, kv_min=0, kv_max=2048, new_min=1, new_max=2048, page=32,
             pad=777, lens=12),
        # the FP32 products of the fused decode + GEMM at a decode batch of 16
        dict(name="rope_step", op="rope", tokens=16, q_heads=32, kv_heads=8, dim=128, rot=128, dtype="fp32",
             norm=True, inter=False, far=131072),
        # a prompt's BF16 queries and keys, strided out of one fused buffer
        dict(name="rope_prompt", op="rope", tokens=8191, q_heads=32, kv_heads=8, dim=128, rot=128, dtype="bf16",
             norm=True, inter=False, far=8192),
        # one decode step's keys and values, FP32 from the fused GEMM
        dict(name="cache_step", op="cache", tokens=64, kv_heads=8, dim=128, page=16, dtype="fp32", pad=3),
        # a prompt of odd length, narrow heads
        dict(name="cache_narrow", op="cache", tokens=2047, kv_heads=5, dim=64, page=64, dtype="bf16", pad=0),
        # the largest prompt chunk taken in by one step
        dict(name="cache_prompt", op="cache", tokens=16384, kv_heads=8, dim=128, page=64, dtype="bf16", pad=0),
        # a single request's token: latency
        dict(name="attend_one", op="attend", reqs=1, q_min=1, q_max=1, kv_min=1017, kv_max=1017, q_heads=32,
             kv_heads=8, dim=128, page=16, causal=True, window=0, lens=21),
        # a decode batch of ragged lengths
        dict(name="attend_batch", op="attend", reqs=64, q_min=1, q_max=1, kv_min=256, kv_max=16384, q_heads=32,
             kv_heads=8, dim=128, page=16, causal=True, window=0, lens=22),
        # two long documents, read token by token (an odd length and a full one)
        dict(name="attend_long", op="attend", reqs=2, q_min=1, q_max=1, kv_min=98301, kv_max=131072, q_heads=32,
             kv_heads=8, dim=128, page=64, causal=True, window=0, lens=23),
        # prompt chunks of odd lengths beside decode tokens, narrow heads, groups of three
        dict(name="attend_mixed", op="attend", reqs=9, q_min=1, q_max=1023, kv_min=1, kv_max=8192, q_heads=24,
             kv_heads=8, dim=64, page=32, causal=True, window=2048, lens=24),
        # a whole prompt
        dict(name="attend_prompt", op="attend", reqs=1, q_min=8192, q_max=8192, kv_min=8192, kv_max=8192, q_heads=32,
             kv_heads=8, dim=128, page=64, causal=True, window=0, lens=25),
    ]


def _log_int(rng, lo, hi):
    """An integer of [lo, hi], spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(max(lo, 1)), math.log(max(hi, 1))))))))


def draw(rng):
    op = rng.choice(("extend", "rope", "cache", "attend", "attend", "attend"))
    lens = rng.randrange(1 << 30)
    if op == "extend":
        prompts = rng.random() < 0.5
        return dict(op=op, reqs=_log_int(rng, 1, 600), kv_min=0, kv_max=_log_int(rng, 16, 8192), new_min=0,
                    new_max=_log_int(rng, 2, 1500) if prompts else rng.randint(1, 4), page=rng.choice((16, 32, 64, 128)),
                    pad=rng.choice((0, rng.randint(1, 900))), lens=lens)
    if op == "rope":
        dim = rng.choice((64, 128, 128, 256))
        kv = rng.choice((1, 2, 5, 8))
        return dict(op=op, tokens=_log_int(rng, 1, 4000), q_heads=kv * rng.choice((1, 3, 4, 8)) if dim < 256 else 16,
                    kv_heads=kv, dim=dim, rot=rng.choice((dim, dim, dim // 2, 8)), dtype=rng.choice(("fp32", "bf16")),
                    norm=rng.random() < 0.75, inter=rng.random() < 0.4, far=_log_int(rng, 64, 1 << 20))
    if op == "cache":
        return dict(op=op, tokens=_log_int(rng, 1, 12000), kv_heads=rng.choice((1, 2, 5, 8)), dim=rng.choice((64, 128)),
                    page=rng.choice((16, 32, 64, 128)), dtype=rng.choice(("fp32", "bf16")),
                    pad=rng.choice((0, rng.randint(1, 30))))
    kv = rng.choice((1, 2, 4, 8))
    shape = dict(q_heads=kv * rng.choice((1, 2, 3, 4, 8)), kv_heads=kv, dim=rng.choice((64, 128, 128)),
                 page=rng.choice((16, 32, 64, 128)), lens=lens)
    kind = rng.choice(("step", "step", "few", "chunk", "whole"))
    if kind == "step":  # single tokens
        reqs = _log_int(rng, 1, 100)
        return dict(op=op, reqs=reqs, q_min=1, q_max=1, kv_min=1, kv_max=_log_int(rng, 64, min(100000, 600000 // reqs)),
                    causal=True, window=rng.choice((0, 0, 0, 1024)), **shape)
    if kind == "few":  # a few drafted tokens of each request
        return dict(op=op, reqs=_log_int(rng, 1, 60), q_min=1, q_max=rng.randint(2, 8), kv_min=2,
                    kv_max=_log_int(rng, 64, 8000), causal=True, window=0, **shape)
    if kind == "chunk":  # prompt chunks over a longer context
        return dict(op=op, reqs=rng.randint(1, 6), q_min=1, q_max=_log_int(rng, 16, 1500), kv_min=16,
                    kv_max=_log_int(rng, 1500, 9000), causal=True, window=rng.choice((0, 0, 512)), **shape)
    # whole prompts, or an encoder's states attended without a mask
    n = _log_int(rng, 2, 3000)
    return dict(op=op, reqs=rng.randint(1, 3), q_min=n, q_max=n, kv_min=n, kv_max=n, causal=rng.random() < 0.7,
                window=0, **shape)


def _lengths(case):
    """Per request (new or query tokens, cached tokens before or in all)."""
    rng = random.Random(case["lens"])
    out = []
    for _ in range(case["reqs"]):
        if case["op"] == "extend":
            out.append((_log_int(rng, case["new_min"], case["new_max"]) if case["new_max"] > 1 else
                        rng.randint(case["new_min"], case["new_max"]), rng.randint(case["kv_min"], case["kv_max"])))
        else:
            q = _log_int(rng, case["q_min"], case["q_max"])
            out.append((q, max(q, rng.randint(case["kv_min"], case["kv_max"]))))
    return out


def _visible(case, q, kv):
    """Pairs of a query and a key that its mask leaves, for one request."""
    if not case["causal"]:
        return q * kv
    w = case["window"] or (1 << 60)
    return sum(min(kv - q + i + 1, w) for i in range(q))


def work(case):
    op = case["op"]
    if op == "extend":
        lens = _lengths(case)
        tokens = sum(n for n, _ in lens) + case["pad"]
        fresh = sum(-(-(n + kv) // case["page"]) - -(-kv // case["page"]) for n, kv in lens)
        return {"bytes": case["reqs"] * 16 + tokens * 12 + fresh * 8, "flops": 0}
    if op == "rope":
        n = case["tokens"] * (case["q_heads"] + case["kv_heads"]) * case["dim"]
        size = 4 if case["dtype"] == "fp32" else 2
        return {"bytes": n * (size + 2) + case["tokens"] * 4, "flops": n * 7}
    if op == "cache":
        n = 2 * case["tokens"] * case["kv_heads"] * case["dim"]
        size = 4 if case["dtype"] == "fp32" else 2
        return {"bytes": n * (size + 2) + 2 * (n * 9 // 16) + case["tokens"] * 16, "flops": n * 3}
    nbytes = flops = 0
    for q, kv in _lengths(case):
        seen = kv if not (case["causal"] and case["window"]) else min(kv, case["window"] + q - 1)
        nbytes += seen * case["kv_heads"] * (case["dim"] * 9 // 8) + 4 * q * case["q_heads"] * case["dim"]
        flops += 4 * case["dim"] * case["q_heads"] * _visible(case, q, kv)
    return {"bytes": nbytes, "flops": flops}


# ------------------------------------------------------------------ inputs

def _gen(seed, salt):
    g = torch.Generator(device="cuda")
    g.manual_seed(1000003 * seed + salt)
    return g


def _randn(shape, g):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)


def _keys(shape, g):
    """Keys as models have them: a few channels much larger than the rest."""
    k = _randn(shape, g)
    d = shape[-1]
    k[..., 3] *= 6.0
    k[..., d // 2 + 5] *= 9.0
    return k


def _page_bytes(case):
    return case["page"] * case["dim"] * 9 // 8


def _own():
    from entropy_decoding_b200 import df11
    return df11


def prepare(case, seed):
    return globals()["_prepare_" + case["op"]](case, seed)


def _prepare_extend(case, seed):
    lens = _lengths(case)
    page, reqs = case["page"], case["reqs"]
    tokens = sum(n for n, _ in lens) + case["pad"]
    width = max(-(-(n + kv) // page) for n, kv in lens) + 3
    held = sum(-(-kv // page) for _, kv in lens)
    fresh = sum(-(-(n + kv) // page) for n, kv in lens) - held
    ids = torch.randperm(held + fresh + 5, generator=_gen(seed, 1), device="cuda").to(torch.int32)
    table = torch.full((reqs, width), -1, dtype=torch.int32, device="cuda")
    kv = torch.tensor([b for _, b in lens], dtype=torch.int32, device="cuda")
    cols = torch.arange(width, device="cuda")
    mine = cols[None, :] < ((kv + page - 1) // page)[:, None]
    table[mine] = ids[:held]
    i32 = dict(dtype=torch.int32, device="cuda")
    return dict(op="extend", page=page, reqs=reqs, tokens=max(tokens, 1), width=width, kv=kv,
                new=torch.tensor([a for a, _ in lens], **i32), table=table, free=ids[held:].contiguous(),
                n_free=torch.tensor([fresh + 5], **i32), kv_out=torch.zeros(reqs, **i32),
                q_start=torch.zeros(reqs + 1, **i32), slots=torch.zeros(max(tokens, 1), dtype=torch.int64, device="cuda"),
                positions=torch.zeros(max(tokens, 1), **i32), n_free_out=torch.zeros(1, **i32))


def _prepare_rope(case, seed):
    g = _gen(seed, 2)
    t, hq, hk, d = case["tokens"], case["q_heads"], case["kv_heads"], case["dim"]
    dt = torch.float32 if case["dtype"] == "fp32" else torch.bfloat16
    width = (hq + 2 * hk) * d  # queries, keys and values of a token side by side
    x = (_randn((t, width), g) * 1.7).to(dt)
    wq, wk = [(1 + 0.2 * _randn((d,), g)).to(torch.bfloat16) for _ in range(2)]
    pos = torch.randint(0, case["far"], (t,), generator=g, device="cuda", dtype=torch.int32)
    rot = case["rot"]
    freq = 500000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)
    out = dict(dtype=torch.bfloat16, device="cuda")
    return dict(op="rope", tokens=t, hq=hq, hk=hk, d=d, rot=rot, inter=case["inter"], dtype=case["dtype"], x=x,
                width=width, wq=wq if case["norm"] else None, wk=wk if case["norm"] else None, pos=pos, freq=freq,
                eps=1e-6, q_out=torch.zeros((t, hq, d), **out), k_out=torch.zeros((t, hk, d), **out))


def _prepare_cache(case, seed):
    g = _gen(seed, 3)
    t, h, d, page = case["tokens"], case["kv_heads"], case["dim"], case["page"]
    dt = torch.float32 if case["dtype"] == "fp32" else torch.bfloat16
    n_pages = -(-t // page) + 4
    slots = torch.randperm(n_pages * page, generator=g, device="cuda")[:t].contiguous()
    if t > page:  # in earnest: whole pages in some order, a prompt's tokens in order within them
        order = torch.randperm(n_pages, generator=g, device="cuda")
        i = torch.arange(t, device="cuda")
        slots = order[i // page] * page + i % page
    pad = case["pad"]
    if pad:
        slots = torch.cat([slots, torch.full((pad,), -1, dtype=slots.dtype, device="cuda")])
    t += pad
    kv = torch.cat([_keys((t, h, d), g), _randn((t, h, d), g) * 0.6], dim=1).to(dt)  # (t, 2 h, d)
    pages = torch.zeros((n_pages, h, _page_bytes(case)), dtype=torch.uint8, device="cuda")
    out = dict(dtype=torch.bfloat16, device="cuda")
    s = dict(op="cache", tokens=t, h=h, d=d, page=page, kv=kv, dtype=case["dtype"], slots=slots, pages=pages,
             gk=0.5, gv=0.25, k_out=torch.zeros((t, h, d), **out), v_out=torch.zeros((t, h, d), **out))
    if own:
        s["cache"] = _own().Kv4Cache(pages.data_ptr(), n_pages, page, h, d, s["gk"], s["gv"])
    return s


def _prepare_attend(case, seed):
    g = _gen(seed, 4)
    lens = _lengths(case)
    hq, h, d, page = case["q_heads"], case["kv_heads"], case["dim"], case["page"]
    counts = [-(-kv // page) for _, kv in lens]
    n_pages, width = sum(counts) + 2, max(counts) + 1
    ids = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
    table = torch.full((len(lens), width), -1, dtype=torch.int32, device="cuda")
    at = 0
    for r, c in enumerate(counts):
        table[r, :c] = ids[at:at + c]
        at += c
    gk, gv = 0.5, 0.25
    pages = torch.empty((n_pages, h, _page_bytes(case)), dtype=torch.uint8, device="cuda")
    step = max(1, (1 << 26) // (page * h * d))
    for p0 in range(0, n_pages, step):  # page by page, as a server fills them
        n = min(step, n_pages - p0)
        slots = torch.arange(p0 * page, (p0 + n) * page, device="cuda")
        _write_pages(pages, page, d, slots, _keys((n * page, h, d), g).to(torch.bfloat16),
                     (_randn((n * page, h, d), g) * 0.6).to(torch.bfloat16), gk, gv)
    starts = [0]
    for q, _ in lens:
        starts.append(starts[-1] + q)
    q = (_randn((starts[-1], hq, d), g) * 0.6).to(torch.bfloat16)
    i32 = dict(dtype=torch.int32, device="cuda")
    s = dict(op="attend", hq=hq, h=h, d=d, page=page, reqs=len(lens), width=width, pages=pages, table=table, q=q,
             lens=lens, starts=starts, q_start=torch.tensor(starts, **i32),
             kv_lens=torch.tensor([kv for _, kv in lens], **i32), causal=case["causal"], window=case["window"],
             scale=d ** -0.5, gk=gk, gv=gv, max_q=max(a for a, _ in lens), o=torch.zeros_like(q),
             lse=torch.zeros((starts[-1], hq), dtype=torch.float32, device="cuda"))
    if own:
        df11 = _own()
        s["cache"] = df11.Kv4Cache(pages.data_ptr(), n_pages, page, h, d, gk, gv)
        need = df11.df11_kv4_attention_workspace_bytes(s["cache"], hq, len(lens), starts[-1], s["max_q"])
        s["ws"] = torch.zeros(max(need, 16), dtype=torch.uint8, device="cuda")
    return s


# ------------------------------------------------------------------ passes

def run(state):
    return globals()[("_own_" if own else "_plain_") + state["op"]](state)


def _stream():
    return torch.cuda.current_stream().cuda_stream


def _own_extend(s):
    _own().df11_kv_extend(s["kv"].data_ptr(), s["new"].data_ptr(), s["reqs"], s["free"].data_ptr(), s["n_free"].data_ptr(),
                          s["table"].data_ptr(), s["width"], s["page"], s["kv_out"].data_ptr(), s["q_start"].data_ptr(),
                          s["slots"].data_ptr(), s["positions"].data_ptr(), s["tokens"], s["n_free_out"].data_ptr(),
                          stream=_stream())
    return s["table"], s["kv_out"], s["q_start"], s["slots"], s["positions"], s["n_free_out"]


def _own_rope(s):
    x, d = s["x"], s["d"]
    size = x.element_size()
    _own().df11_qk_norm_rope(
        (x.data_ptr(), s["width"], s["wq"].data_ptr() if s["wq"] is not None else 0, s["q_out"].data_ptr(), s["hq"] * d,
         s["hq"]),
        (x.data_ptr() + s["hq"] * d * size, s["width"], s["wk"].data_ptr() if s["wk"] is not None else 0,
         s["k_out"].data_ptr(), s["hk"] * d, s["hk"]),
        s["tokens"], d, s["pos"].data_ptr(), s["freq"].data_ptr(), s["rot"], interleaved=s["inter"], eps=s["eps"],
        dtype=s["dtype"], stream=_stream())
    return s["q_out"], s["k_out"]


def _own_cache(s):
    df11, kv, st = _own(), s["kv"], _stream()
    row = 2 * s["h"] * s["d"]
    df11.df11_kv4_append(s["cache"], kv.data_ptr(), row, kv.data_ptr() + s["h"] * s["d"] * kv.element_size(), row,
                         s["slots"].data_ptr(), s["tokens"], dtype=s["dtype"], stream=st)
    df11.df11_kv4_gather(s["cache"], s["slots"].data_ptr(), s["tokens"], s["k_out"].data_ptr(), s["v_out"].data_ptr(),
                         stream=st)
    return s["k_out"], s["v_out"]


def _own_attend(s):
    row = s["hq"] * s["d"]
    _own().df11_kv4_attention(s["cache"], s["q"].data_ptr(), row, s["o"].data_ptr(), row, s["hq"], s["q_start"].data_ptr(),
                              s["kv_lens"].data_ptr(), s["table"].data_ptr(), s["reqs"], s["width"], s["starts"][-1],
                              s["max_q"], s["scale"], s["ws"].data_ptr(), s["ws"].numel(), causal=s["causal"],
                              window=s["window"], lse_ptr=s["lse"].data_ptr(), stream=_stream())
    return s["o"], s["lse"]


# ------------------------------------------------------------------ plain forms

def _plain_extend(s):
    page, kv, new = s["page"], s["kv"].long(), s["new"].long()
    before, after = (kv + page - 1) // page, (kv + new + page - 1) // page
    fresh = after - before
    first = torch.cumsum(fresh, 0) - fresh
    n_free = s["n_free"].long()
    cols = torch.arange(s["width"], device=kv.device)[None, :]
    taken = first[:, None] + cols - before[:, None]
    grows = (cols >= before[:, None]) & (cols < after[:, None])
    at = (n_free - 1 - taken).clamp(0, s["free"].numel() - 1)
    table = torch.where(grows, s["free"][at], s["table"])
    ends = torch.cumsum(new, 0)
    q_start = torch.cat([torch.zeros_like(ends[:1]), ends])
    t = torch.arange(s["tokens"], device=kv.device)
    req = torch.searchsorted(ends, t, right=True)
    live = req < s["reqs"]
    req = req.clamp(max=s["reqs"] - 1)
    pos = torch.where(live, kv[req] + t - q_start[req], torch.zeros_like(t))
    slots = torch.where(live, table[req, pos // page].long() * page + pos % page, torch.full_like(t, -1))
    return (table, (kv + new).int(), q_start.int(), slots, pos.int(), (n_free - fresh.sum()).int())


def _plain_rope(s):
    hq, hk, d, rot = s["hq"], s["hk"], s["d"], s["rot"]
    angle = s["pos"].double()[:, None] * s["freq"][None, :]
    cos, sin = angle.cos().float()[:, None, :], angle.sin().float()[:, None, :]
    outs = []
    for x, w in ((s["x"][:, :hq * d], s["wq"]), (s["x"][:, hq * d:(hq + hk) * d], s["wk"])):
        x = x.float().reshape(s["tokens"], -1, d)
        if w is not None:
            x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + s["eps"]) * w.float()
        a, b = (x[..., :rot:2], x[..., 1:rot:2]) if s["inter"] else (x[..., :rot // 2], x[..., rot // 2:rot])
        y = x.clone()
        if s["inter"]:
            y[..., :rot:2], y[..., 1:rot:2] = a * cos - b * sin, b * cos + a * sin
        else:
            y[..., :rot // 2], y[..., rot // 2:rot] = a * cos - b * sin, b * cos + a * sin
        outs.append(y.to(torch.bfloat16))
    return tuple(outs)


def _quantize(x, g):
    """BF16 (t, h, d) -> 4-bit codes (t, h, d) and E4M3 scale bytes (t, h, d / 16)."""
    x = x.to(torch.bfloat16).float()
    x = x.reshape(*x.shape[:-1], -1, 16)
    s = ((x.abs().amax(-1) / 6.0) / g).clamp(max=448.0).to(torch.float8_e4m3fn)
    step = (s.float() * g)[..., None]
    a = (x.abs() / step).nan_to_num(0.0, posinf=6.0)
    # thresholds between the levels; a tie goes to the level of even mantissa
    code = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))
    code = code | ((x < 0).to(torch.uint8) << 3)
    return code.flatten(-2), s.view(torch.uint8)


def _views(pages, page, d):
    """K codes, K scales, V codes, V scales of the pages (strided views)."""
    n, h, size = pages.shape
    kc, ks = page * d // 2, page * d // 16
    return (pages[..., :kc].view(n, h, page, d // 2), pages[..., kc:kc + ks].view(n, h, page, d // 16),
            pages[..., kc + ks:2 * kc + ks].view(n, h, page // 4, d // 16, 4, 8),
            pages[..., 2 * kc + ks:].view(n, h, d // 16, page))


def _write_pages(pages, page, d, slots, k, v, gk, gv):
    at, off = slots // page, slots % page
    kcodes, kscales, vcodes, vscales = _views(pages, page, d)
    (ck, sk), (cv, sv) = _quantize(k, gk), _quantize(v, gv)
    kcodes[at, :, off] = ck[..., 0::2] | (ck[..., 1::2] << 4)
    kscales[at, :, off] = sk
    packed = cv[..., 0::2] | (cv[..., 1::2] << 4)
    vcodes[at, :, off // 4, :, off % 4] = packed.unflatten(-1, (d // 16, 8))
    vscales[at, :, :, off] = sv


def _read_codes(codes, scales, g):
    """Bytes (..., d / 2) and scale bytes (..., d / 16) -> the values, FP32."""
    table = torch.tensor([v for v in LEVELS] + [-v for v in LEVELS], dtype=torch.float32, device=codes.device)
    x = torch.stack([table[(codes & 15).int()], table[(codes >> 4).int()]], dim=-1).flatten(-2)
    s = scales.contiguous().view(torch.float8_e4m3fn).float() * g
    return (x.unflatten(-1, (-1, 16)) * s[..., None]).flatten(-2)


def _plain_cache(s):
    live = s["slots"] >= 0
    slots, h, d, page = s["slots"][live], s["h"], s["d"], s["page"]
    _write_pages(s["pages"], page, d, slots, s["kv"][live, :h], s["kv"][live, h:], s["gk"], s["gv"])
    kcodes, kscales, vcodes, vscales = _views(s["pages"], page, d)
    at, off = slots // page, slots % page
    s["k_out"][live] = _read_codes(kcodes[at, :, off], kscales[at, :, off], s["gk"]).to(torch.bfloat16)
    s["v_out"][live] = _read_codes(vcodes[at, :, off // 4, :, off % 4].flatten(-2), vscales[at, :, :, off],
                                   s["gv"]).to(torch.bfloat16)
    return s["k_out"], s["v_out"]


def _plain_attend(s):
    h, d, page, group = s["h"], s["d"], s["page"], s["hq"] // s["h"]
    views = _views(s["pages"], page, d)
    for r, (n, kv) in enumerate(s["lens"]):
        t0 = s["starts"][r]
        ids = s["table"][r, :-(-kv // page)].long()
        kc, ks, vc, vs = [x[ids] for x in views]
        k = _read_codes(kc, ks, s["gk"]).transpose(0, 1).reshape(h, -1, d)[:, :kv]
        v = _read_codes(vc.transpose(3, 4).flatten(2, 3).flatten(-2), vs.transpose(2, 3), s["gv"])
        v = v.transpose(0, 1).reshape(h, -1, d)[:, :kv]
        q = s["q"][t0:t0 + n].float().reshape(n, h, group, d).permute(1, 2, 0, 3)  # (h, group, n, d)
        rows = torch.arange(n, device=q.device)[:, None] + (kv - n)
        cols = torch.arange(kv, device=q.device)[None, :]
        keep = (cols <= rows) if s["causal"] else torch.ones((n, kv), dtype=torch.bool, device=q.device)
        if s["causal"] and s["window"]:
            keep = keep & (cols > rows - s["window"])
        heads = 1 if n > 64 else h
        for i in range(0, h, heads):
            sc = torch.matmul(q[i:i + heads], k[i:i + heads, None].transpose(-1, -2)) * s["scale"]
            sc = sc.masked_fill(~keep, float("-inf"))
            top = sc.amax(-1, keepdim=True)
            p = torch.exp(sc - torch.where(top == float("-inf"), torch.zeros_like(top), top))
            total = p.sum(-1, keepdim=True)
            o = torch.matmul(p, v[i:i + heads, None]) / torch.where(total == 0, torch.ones_like(total), total)
            s["o"][t0:t0 + n].view(n, h, group, d)[:, i:i + heads] = o.permute(2, 0, 1, 3).to(torch.bfloat16)
            lse = (top + torch.log(total))[..., 0]
            s["lse"][t0:t0 + n].view(n, h, group)[:, i:i + heads] = lse.permute(2, 0, 1)
    return s["o"], s["lse"]


# ------------------------------------------------------------------ the definitions, in 64 bits

def exact(case, seed):
    state = prepare(case, seed)
    return globals()["_exact_" + case["op"]](state)


def _exact_extend(s):
    """Request by request, token by token, on the host."""
    page = s["page"]
    table, free = s["table"].cpu().tolist(), s["free"].cpu().tolist()[:int(s["n_free"].item())]
    kv_out, q_start, slots, positions = [], [0], [], []
    for r, (kv, new) in enumerate(zip(s["kv"].cpu().tolist(), s["new"].cpu().tolist())):
        for p in range(kv, kv + new):
            if p % page == 0:
                table[r][p // page] = free.pop()
            slots.append(table[r][p // page] * page + p % page)
            positions.append(p)
        kv_out.append(kv + new)
        q_start.append(len(slots))
    pad = s["tokens"] - len(slots)
    t = torch.tensor
    return (t(table), t(kv_out), t(q_start), t(slots + [-1] * pad), t(positions + [0] * pad), t([len(free)]))


def _exact_rope(s):
    """Each pair as a complex number turned by exp(i angle)."""
    hq, hk, d, rot = s["hq"], s["hk"], s["d"], s["rot"]
    turn = torch.exp(1j * torch.outer(s["pos"].double(), s["freq"]))[:, None, :]
    full = s["x"].double().unflatten(1, (hq + 2 * hk, d))
    outs = []
    for x, w in ((full[:, :hq], s["wq"]), (full[:, hq:hq + hk], s["wk"])):
        if w is not None:
            x = x / torch.sqrt(torch.linalg.vector_norm(x, dim=-1, keepdim=True) ** 2 / d + s["eps"]) * w.double()
        head, tail = x[..., :rot], x[..., rot:]
        pairs = head.unflatten(-1, (rot // 2, 2)) if s["inter"] else head.unflatten(-1, (2, rot // 2)).transpose(-1, -2)
        z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn)
        z = z.flatten(-2) if s["inter"] else z.transpose(-1, -2).flatten(-2)
        outs.append(torch.cat([z, tail], dim=-1))
    return tuple(outs)


def _nearest(x, grid):
    """The entry of the ascending grid nearest to x; a tie goes to the entry of even index."""
    hi = torch.searchsorted(grid, x).clamp(1, grid.numel() - 1)
    lo = hi - 1
    dl, dh = x - grid[lo], grid[hi] - x
    up = (dh < dl) | ((dh == dl) & (hi % 2 == 0))
    return torch.where(up, grid[hi], grid[lo])


def _exact_cache(s):
    # the non-negative E4M3 values in order of their bytes 0 .. 126
    scales = [(m / 8) * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7) for e in range(16) for m in range(8)][:127]
    scales = torch.tensor(scales, dtype=torch.float64, device="cuda")
    levels = torch.tensor(LEVELS, dtype=torch.float64, device="cuda")
    outs = []
    for x, g in ((s["kv"][:, :s["h"]], s["gk"]), (s["kv"][:, s["h"]:], s["gv"])):
        x = x.to(torch.bfloat16).double().unflatten(-1, (s["d"] // 16, 16))
        unit = _nearest(x.abs().amax(-1, keepdim=True) / (6 * g), scales) * g
        level = _nearest(x.abs() / torch.where(unit == 0, torch.ones_like(unit), unit), levels)
        value = (torch.sign(x) * level * unit).flatten(-2)
        outs.append(torch.where((s["slots"] >= 0)[:, None, None], value, torch.zeros_like(value)))
    return tuple(outs)


def _exact_attend(s):
    """Head by head, the values of a byte's two codes from a table of 256."""
    h, d, page, group = s["h"], s["d"], s["page"], s["hq"] // s["h"]
    signed = [v for v in LEVELS] + [-v for v in LEVELS]
    pair = torch.tensor([[signed[b & 15], signed[b >> 4]] for b in range(256)], dtype=torch.float64, device="cuda")
    e4m3 = torch.arange(256, device="cuda", dtype=torch.int32)
    mant, ex = (e4m3 & 7).double(), ((e4m3 >> 3) & 15)
    unit = torch.where(ex == 0, mant / 8 * 2.0 ** -6, (1 + mant / 8) * torch.pow(2.0, (ex - 7).double()))
    kc, ks = page * d // 2, page * d // 16
    o = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros(s["lse"].shape, dtype=torch.float64, device="cuda")
    for r, (n, kv) in enumerate(s["lens"]):
        t0 = s["starts"][r]
        ids = s["table"][r, :-(-kv // page)].long()
        i = torch.arange(n, device="cuda")[:, None]
        j = torch.arange(kv, device="cuda")[None, :]
        hidden = torch.zeros((n, kv), dtype=torch.bool, device="cuda")
        if s["causal"]:
            hidden = j - i > kv - n
            if s["window"]:
                hidden = hidden | (j - i <= kv - n - s["window"])
        for head in range(h):
            b = s["pages"][ids, head]
            m = b.shape[0]
            k = pair[b[:, :kc].long()].view(m * page, d // 16, 16)
            k = (k * unit[b[:, kc:kc + ks].long()].view(m * page, d // 16, 1)).view(-1, d)[:kv] * s["gk"]
            v = pair[b[:, kc + ks:2 * kc + ks].long()].view(m, page // 4, d // 16, 4, 16)
            v = v * unit[b[:, 2 * kc + ks:].long()].view(m, d // 16, page // 4, 4).permute(0, 2, 1, 3)[..., None]
            v = v.transpose(2, 3).reshape(m * page, d)[:kv] * s["gv"]
            for g in range(group):
                c = head * group + g
                sc = (s["q"][t0:t0 + n, c].double() @ k.T) * s["scale"]
                sc[hidden] = -math.inf
                z = torch.logsumexp(sc, dim=-1)
                lse[t0:t0 + n, c] = z
                w = torch.exp(sc - z[:, None])
                w[torch.isneginf(z)] = 0
                o[t0:t0 + n, c] = w @ v
    return o, lse
