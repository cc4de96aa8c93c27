"""The serving operators on the GPU against their 64-bit forms (serve_ref):
pages and slots, norm and rotation, the 4-bit cache, attention over it, and a
whole attention step with the fused decode + GEMM around it, eager, on another
stream and captured into a graph."""
import numpy as np
import pytest
import torch

import serve_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def df11():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from entropy_decoding_b200 import build
    build.build()
    from entropy_decoding_b200 import df11 as mod
    return mod


def dev(x, dtype):
    return torch.as_tensor(np.asarray(x)).to(dtype).cuda()


def word():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def stream():
    return torch.cuda.current_stream().cuda_stream


# ------------------------------------------------------------------ pages, slots, positions

def run_extend(df11, kv, new, free, n_free, table, page, max_tokens, guard=7):
    """Outputs between guard words; returns the reference's six results and the error word."""
    i32 = torch.int32
    n, w = len(kv), len(table[0]) if len(table) else 0
    bufs = dict(table=dev(np.array(table).reshape(-1), i32), kv_out=torch.full((n + guard,), 77, dtype=i32, device="cuda"),
                q_start=torch.full((n + 1 + guard,), 77, dtype=i32, device="cuda"),
                slots=torch.full((max_tokens + guard,), 77, dtype=torch.int64, device="cuda"),
                pos=torch.full((max_tokens + guard,), 77, dtype=i32, device="cuda"),
                nf=torch.full((1 + guard,), 77, dtype=i32, device="cuda"))
    kvd, newd = dev(np.array(kv, np.int64), i32), dev(np.array(new, np.int64), i32)
    fd, nfd = dev(np.array(list(free) + [0]), i32), dev([n_free], i32)
    err = word()
    df11.df11_kv_extend(kvd.data_ptr(), newd.data_ptr(), n, fd.data_ptr(), nfd.data_ptr(), bufs["table"].data_ptr(), w,
                        page, bufs["kv_out"].data_ptr(), bufs["q_start"].data_ptr(), bufs["slots"].data_ptr(),
                        bufs["pos"].data_ptr(), max_tokens, bufs["nf"].data_ptr(), err.data_ptr(), stream())
    torch.cuda.synchronize()
    out = {k: v.cpu().tolist() for k, v in bufs.items()}
    for k, size in (("kv_out", n), ("q_start", n + 1), ("slots", max_tokens), ("pos", max_tokens), ("nf", 1)):
        assert out[k][size:] == [77] * guard, k
    return ([out["table"][r * w:(r + 1) * w] for r in range(n)], out["kv_out"][:n], out["q_start"][:n + 1],
            out["slots"][:max_tokens], out["pos"][:max_tokens], out["nf"][0]), int(err.item())


@pytest.mark.parametrize("reqs,page,kv_max,new_max,pad", [
    (1, 16, 0, 1, 0), (1, 128, 300, 700, 5), (3, 16, 40, 0, 4), (128, 16, 900, 1, 0), (511, 32, 100, 3, 1),
    (512, 64, 90, 2, 511), (513, 16, 64, 5, 513), (1500, 32, 70, 4, 100), (40, 64, 500, 900, 33), (2, 16, 31, 4000, 0)])
def test_extend(df11, reqs, page, kv_max, new_max, pad):
    g = np.random.default_rng(reqs + page)
    kv, new = g.integers(0, kv_max + 1, reqs), g.integers(0, new_max + 1, reqs)
    kv[g.random(reqs) < 0.2] = 0
    kv[g.random(reqs) < 0.2] = page  # full pages
    w = int(-(-(kv + new).max() // page)) + 2
    held = -(-kv // page)
    fresh = int((-(-(kv + new) // page) - held).sum())
    ids = g.permutation(int(held.sum()) + fresh + 3)
    table, at = np.full((reqs, w), -7), 0
    for r in range(reqs):
        table[r, :held[r]] = ids[at:at + held[r]]
        at += held[r]
    free = ids[at:]
    max_tokens = int(new.sum()) + pad
    got, err = run_extend(df11, kv, new, free, len(free), table, page, max_tokens)
    want = ref.extend(kv, new, free, len(free), table, page, max_tokens)
    assert err == 0
    for name, a, b in zip(("table", "kv_out", "q_start", "slots", "positions", "n_free"), got, want):
        assert a == b, name


def test_extend_without_requests_is_padding(df11):
    got, err = run_extend(df11, [], [], [3], 1, [], 16, 600)
    assert err == 0 and got == ([], [], [0], [-1] * 600, [0] * 600, 1)


def test_extend_reports_what_does_not_fit(df11):
    P, A = df11.DEV_ERR_PAGES, df11.DEV_ERR_AUX
    # the stack holds one page, two are needed: the second request's rows have no slot
    got, err = run_extend(df11, [0, 0], [3, 2], [5], 1, [[-1], [-1]], 16, 5)
    assert err == P and got[3] == [80, 81, 82, -1, -1] and got[5] == 0
    # a row of the table is too short
    got, err = run_extend(df11, [14], [4], [5, 6], 2, [[9]], 16, 4)
    assert err == P and got[3] == [9 * 16 + 14, 9 * 16 + 15, -1, -1]
    # a held page that is not there
    got, err = run_extend(df11, [14], [1], [5], 1, [[-1, -1]], 16, 1)
    assert err == P and got[3] == [-1]
    # negative lengths count as 0
    got, err = run_extend(df11, [-5, 0], [1, -9], [5, 6], 2, [[-1], [-1]], 16, 2)
    assert err == A and got[1] == [1, 0] and got[2] == [0, 1, 1] and got[3] == [6 * 16, -1]
    # more rows than there is room for: nothing is written past it, q_start is cut
    got, err = run_extend(df11, [0, 0], [3, 4], [5, 6], 2, [[-1], [-1]], 16, 4)
    assert err & A and got[2] == [0, 3, 4] and got[3] == [96, 97, 98, 80]
    # lengths whose sum passes 32 bits
    big = 2 ** 31 - 1
    got, err = run_extend(df11, [0, 0, 0], [big, big, 5], [1, 2], 2, [[-1]] * 3, 16, 3)
    assert err == A | P and got[2] == [0, 3, 3, 3] and got[3] == [32, 33, 34] and got[5] == 0


def extend_with_limits(kv, new, free, table, page, max_tokens):
    """ref.extend for a table of any width, a stack that may run out and rows past max_tokens."""
    table, stack = [list(map(int, row)) for row in table], list(map(int, free))
    kv_out, q_start, slots, pos, pages = [], [0], [], [], False
    for r, (a, n) in enumerate(zip(map(int, kv), map(int, new))):
        for p in range(a, a + n):
            at, room = p // page, p // page < len(table[r])
            if room and p % page == 0:
                table[r][at] = stack.pop() if stack else -1
            if not room or table[r][at] < 0:
                pages = True
            slots.append(table[r][at] * page + p % page if room and table[r][at] >= 0 else -1)
            pos.append(p)
        kv_out.append(a + n)
        q_start.append(min(len(slots), max_tokens))
    pad, over = max(max_tokens - len(slots), 0), len(slots) > max_tokens
    return (table, kv_out, q_start, (slots + [-1] * pad)[:max_tokens], (pos + [0] * pad)[:max_tokens], len(stack)), pages, over


@pytest.mark.parametrize("reqs,page,new_max", [(2, 16, 60), (40, 16, 50), (700, 32, 90), (5, 128, 1500)])
@pytest.mark.parametrize("short", ["rows", "table", "pages", "all"])
def test_extend_loses_no_page(df11, reqs, page, new_max, short):
    """What does not fit is flagged, every page taken from the stack is in the table all the same, and the next step
    finds it there."""
    g = np.random.default_rng(reqs)
    kv, new = g.integers(0, 3 * page, reqs), g.integers(0, new_max + 1, reqs)
    held = -(-kv // page)
    w = int(-(-(kv + new).max() // page)) + 1
    if short in ("table", "all"):
        w = max(int(held.max()), w // 2)
    ids = g.permutation(int(held.sum()) + int((-(-(kv + new) // page) - held).sum()) + 2 * reqs)
    table, at = np.full((reqs, w), -7), 0
    for r in range(reqs):
        table[r, :held[r]] = ids[at:at + held[r]]
        at += held[r]
    free = ids[at:]
    if short in ("pages", "all"):
        free = free[-max(1, int((-(-(kv + new) // page) - held).sum()) // 2):]
    max_tokens = int(new.sum()) // 2 if short in ("rows", "all") else int(new.sum()) + 3
    got, err = run_extend(df11, kv, new, free, len(free), table, page, max_tokens)
    want, pages, over = extend_with_limits(kv, new, free, table, page, max_tokens)
    names = ("table", "kv_out", "q_start", "slots", "positions", "n_free")
    for name, a, b in zip(names, got, want):
        assert a == b, name
    assert err == df11.DEV_ERR_PAGES * pages + df11.DEV_ERR_AUX * over
    taken = [p for row, h in zip(got[0], held) for p in row[h:] if p >= 0]
    assert sorted(taken + list(free[:got[5]])) == sorted(free)
    # one more token for each request
    got2, err2 = run_extend(df11, got[1], [1] * reqs, free, got[5], got[0], page, reqs)
    want2, pages, over = extend_with_limits(want[1], [1] * reqs, free[:want[5]], want[0], page, reqs)
    for name, a, b in zip(names, got2, want2):
        assert a == b, name
    assert err2 == df11.DEV_ERR_PAGES * pages and not over


@pytest.mark.slow
def test_extend_most_rows(df11):
    """As many rows as their count can say (26 GB of slots and positions), all but three of them padding."""
    n = 2 ** 31 - 1
    i32 = dict(dtype=torch.int32, device="cuda")
    slots, pos = torch.full((n,), 7, dtype=torch.int64, device="cuda"), torch.full((n,), 7, **i32)
    kv, new, free, nf, table = (torch.tensor(x, **i32) for x in ([0], [3], [5], [1], [-1]))
    kvo, qs, nfo, err = (torch.zeros(k, **i32) for k in (1, 2, 1, 1))
    df11.df11_kv_extend(kv.data_ptr(), new.data_ptr(), 1, free.data_ptr(), nf.data_ptr(), table.data_ptr(), 1, 16,
                        kvo.data_ptr(), qs.data_ptr(), slots.data_ptr(), pos.data_ptr(), n, nfo.data_ptr(), err.data_ptr(),
                        stream())
    torch.cuda.synchronize()
    assert err.item() == 0 and kvo.item() == 3 and qs.tolist() == [0, 3] and nfo.item() == 0 and table.item() == 5
    assert slots[:3].tolist() == [80, 81, 82] and pos[:3].tolist() == [0, 1, 2]
    for x, want in ((slots, -1), (pos, 0)):
        lo, hi = x[3:].aminmax()
        assert lo.item() == want and hi.item() == want


def test_extend_repeats_and_chains(df11):
    """The same call twice gives the same result; the next step takes the outputs as inputs."""
    i32, page, n = torch.int32, 16, 5
    kv, free, nf = [dev([0, 3, 15, 16, 31], i32)], dev(np.arange(40), i32), [dev([40], i32)]
    table = torch.full((n, 12), -1, dtype=i32, device="cuda")
    for r, c in enumerate([0, 1, 1, 1, 2]):
        for p in range(c):
            table[r, p] = 100 + 10 * r + p
    new = dev([1, 1, 1, 20, 0], i32)
    wt, wkv, wnf = table.cpu().tolist(), [0, 3, 15, 16, 31], 40
    for _ in range(4):
        for _ in range(2):
            qs, slots, pos = (torch.empty(n + 1, dtype=i32, device="cuda"),
                              torch.empty(30, dtype=torch.int64, device="cuda"), torch.empty(30, dtype=i32, device="cuda"))
            ko, no = torch.empty(n, dtype=i32, device="cuda"), torch.empty(1, dtype=i32, device="cuda")
            df11.df11_kv_extend(kv[-1].data_ptr(), new.data_ptr(), n, free.data_ptr(), nf[-1].data_ptr(),
                                table.data_ptr(), 12, page, ko.data_ptr(), qs.data_ptr(), slots.data_ptr(),
                                pos.data_ptr(), 30, no.data_ptr(), stream=stream())
        torch.cuda.synchronize()
        wt, wkv, wqs, wslots, wpos, wnf = ref.extend(wkv, [1, 1, 1, 20, 0], np.arange(40), wnf, wt, page, 30)
        assert table.cpu().tolist() == wt and ko.cpu().tolist() == wkv and qs.cpu().tolist() == wqs
        assert slots.cpu().tolist() == wslots and pos.cpu().tolist() == wpos and no.item() == wnf
        kv.append(ko)
        nf.append(no)


# ------------------------------------------------------------------ norm and rotation

def rope_case(df11, t, hq, hk, d, rot, dtype, norm, inter, far, seed=0, in_place=False, pad=16, scale=1.7, eps=1e-6):
    g = np.random.default_rng(seed + t + hq)
    dt = torch.float32 if dtype == "fp32" else torch.bfloat16
    width = (hq + hk) * d + pad
    x = dev(g.standard_normal((t, width)) * scale, dt)
    ws = [dev(1 + 0.3 * g.standard_normal(d), torch.bfloat16) if norm else None for _ in range(2)]
    pos = g.integers(0, far + 1, t)
    pos[0] = far
    freq = 500000.0 ** (-np.arange(0, max(rot, 2), 2) / max(rot, 2))[:rot // 2]
    posd, freqd = dev(pos, torch.int32), dev(np.append(freq, 0.0), torch.float64)
    x64 = x.double().cpu().numpy()
    outs, want = [], []
    for base, heads, w in ((0, hq, ws[0]), (hq * d, hk, ws[1])):
        xx = x64[:, base:base + heads * d].reshape(t, heads, d)
        want.append(ref.norm_rope(xx, w.double().cpu().numpy() if w is not None else None, pos, freq, rot, inter, eps))
        outs.append(x[:, base:base + heads * d] if in_place else
                    torch.full((t, heads * d + 8), 7.0, dtype=torch.bfloat16, device="cuda"))
    sides = []
    for (base, heads, w), o in zip(((0, hq, ws[0]), (hq * d, hk, ws[1])), outs):
        sides.append((x.data_ptr() + base * x.element_size(), width, w.data_ptr() if norm else 0, o.data_ptr(),
                      width if in_place else heads * d + 8, heads))
    df11.df11_qk_norm_rope(sides[0], sides[1], t, d, posd.data_ptr(), freqd.data_ptr(), rot, interleaved=inter, eps=eps,
                           dtype=dtype, stream=stream())
    torch.cuda.synchronize()
    for o, (y, mag), heads in zip(outs, want, (hq, hk)):
        if not in_place:
            assert (o[:, heads * d:] == 7.0).all()
        got = o[:, :heads * d].double().cpu().numpy().reshape(t, heads, d)
        # sine and cosine within 2^-21 (the angle's remainder rounded to 32 bits, the functions' own last bits, the
        # pair's products and sum); the norm's sum of d squares, root and products within (d / 2 + 8) 2^-24 relative;
        # then one rounding to BF16
        e = mag * ((d / 2 + 8) * 2.0 ** -24 + 2.0 ** -21)
        assert (np.abs(got - y) <= e + 2.0 ** -8 * (np.abs(y) + e)).all()


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("t,hq,hk,d,rot,norm,far", [
    (1, 32, 8, 128, 128, True, 131071), (16, 32, 8, 128, 128, True, 2000000), (7, 5, 1, 64, 64, True, 100),
    (300, 9, 3, 128, 64, True, 8191), (700, 17, 1, 256, 256, True, 4096), (33, 1, 1, 64, 8, False, 2 ** 31 - 1),
    (5, 3, 3, 256, 24, True, 77), (4, 7, 2, 128, 0, True, 9), (601, 32, 8, 128, 128, False, 8192)])
def test_rope(df11, t, hq, hk, d, rot, norm, far, dtype, inter):
    rope_case(df11, t, hq, hk, d, rot, dtype, norm, inter, far)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("t,hq,hk,d", [(1100, 100, 7, 128), (300, 100, 7, 64), (1, 300, 90, 256), (530, 45, 30, 256)])
def test_rope_many_heads(df11, t, hq, hk, d, dtype):
    """More heads than a thread has in flight."""
    rope_case(df11, t, hq, hk, d, d, dtype, True, False, 5000)


def test_rope_in_place(df11):
    rope_case(df11, 65, 6, 2, 128, 128, "bf16", True, False, 4000, in_place=True)
    rope_case(df11, 65, 6, 2, 64, 32, "bf16", True, True, 4000, in_place=True)


def test_rope_extremes(df11):
    """Heads of zeros (eps alone under the root), of tiny and of huge values."""
    rope_case(df11, 9, 4, 2, 128, 128, "fp32", True, False, 50, scale=0.0)
    rope_case(df11, 9, 4, 2, 128, 128, "fp32", True, False, 50, scale=1e-6)
    rope_case(df11, 9, 4, 2, 128, 128, "fp32", True, False, 50, scale=1e12)
    rope_case(df11, 9, 4, 2, 128, 128, "fp32", True, False, 50, scale=1e-3, eps=0.0)


def test_rope_one_side(df11):
    x = torch.randn(5, 256, device="cuda")
    o = torch.zeros(5, 256, dtype=torch.bfloat16, device="cuda")
    pos, freq = dev(np.arange(5), torch.int32), dev(0.1 * np.arange(64), torch.float64)
    y = ref.norm_rope(x.double().cpu().numpy().reshape(5, 2, 128), None, np.arange(5), 0.1 * np.arange(64), 128, False, 0)[0]
    side = (x.data_ptr(), 256, 0, o.data_ptr(), 256, 2)
    for q, k in ((side, None), (None, side)):
        o.zero_()
        df11.df11_qk_norm_rope(q, k, 5, 128, pos.data_ptr(), freq.data_ptr(), 128, stream=stream())
        torch.cuda.synchronize()
        assert np.abs(o.double().cpu().numpy().reshape(5, 2, 128) - y).max() <= 2.0 ** -8 * np.abs(y).max() + 1e-6


def test_rope_absent_side_is_not_read(df11):
    """Of a side without heads no pointer is checked, so none is followed: what it holds is any number."""
    x = torch.randn(5, 256, device="cuda")
    pos, freq = dev(np.arange(5), torch.int32), dev(0.1 * np.arange(64), torch.float64)
    w = dev(1 + 0.1 * np.arange(128) / 128, torch.bfloat16)
    absent = (2, 1, 2, 2, 1, 0)
    outs = []
    for left_out in (None, absent):
        for first in (True, False):
            o = torch.zeros(5, 256, dtype=torch.bfloat16, device="cuda")
            side = (x.data_ptr(), 256, w.data_ptr(), o.data_ptr(), 256, 2)
            q, k = (side, left_out) if first else (left_out, side)
            df11.df11_qk_norm_rope(q, k, 5, 128, pos.data_ptr(), freq.data_ptr(), 128, stream=stream())
            torch.cuda.synchronize()
            outs.append(o)
    assert outs[0].any() and all(torch.equal(o, outs[0]) for o in outs)


# ------------------------------------------------------------------ the cache

def device_cache(df11, c, pages=None):
    pages = torch.from_numpy(c.bytes.copy()).cuda() if pages is None else pages
    h = df11.Kv4Cache(pages.data_ptr(), c.n_pages, c.page, c.heads, c.dim, c.gk, c.gv)
    return h, pages


def some_kv(g, t, h, d, spread=1.0):
    """Values over many binades, with zero blocks, whole levels and their borders among them."""
    x = g.standard_normal((t, h, d)) * np.exp2(g.integers(-6, 7, (t, h, 1)) * spread)
    x[g.random((t, h, d)) < 0.1] = 0
    x.reshape(t, h, -1, 16)[g.random((t, h, d // 16)) < 0.1] = 0
    m = g.random((t, h)) < 0.3
    x[m] = g.integers(-24, 25, (int(m.sum()), d)) / 4.0
    return x.astype(np.float32)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("t,h,d,page,gk,gv", [(1, 1, 64, 16, 1.0, 1.0), (3, 2, 128, 16, 0.5, 2.0 ** -7), (9, 40, 64, 16, 1.0, 0.5), (65, 8, 128, 32, 1.0, 0.013),
                                              (130, 5, 64, 128, 0.37, 1.9), (258, 3, 128, 64, 2.0 ** -12, 64.0)])
def test_append_and_gather(df11, t, h, d, page, gk, gv, dtype):
    g = np.random.default_rng(t + d)
    n_pages = -(-t // page) + 2
    c = ref.Cache(n_pages, page, h, d, gk, gv, fill=0xA5)
    k, v = some_kv(g, t, h, d), some_kv(g, t, h, d, 0.5)
    slots = g.permutation(n_pages * page)[:t]
    slots[g.random(t) < 0.1] = -1
    handle, pages = device_cache(df11, c)
    dt = torch.float32 if dtype == "fp32" else torch.bfloat16
    kd = torch.full((t, h * d + 16), 3.0, dtype=dt, device="cuda")
    vd = torch.full((t, h * d + 24), 3.0, dtype=dt, device="cuda")
    kd[:, :h * d], vd[:, :h * d] = dev(k.reshape(t, -1), dt), dev(v.reshape(t, -1), dt)
    sd, err = dev(slots, torch.int64), word()
    df11.df11_kv4_append(handle, kd.data_ptr(), h * d + 16, vd.data_ptr(), h * d + 24, sd.data_ptr(), t, dtype=dtype,
                         err_ptr=err.data_ptr(), stream=stream())
    torch.cuda.synchronize()
    c.write(slots, k, v)
    got = pages.cpu().numpy()
    # a zero's sign is the level's only freedom: compare the bytes with the nibbles' negative zeros cleared
    assert err.item() == 0
    codes = page * d // 2

    def canon(b):
        b = b.copy()
        for lo in (0, codes + page * d // 16):
            x = b[..., lo:lo + codes]
            x[(x & 0x0F) == 0x08] &= 0xF0
            x[(x & 0xF0) == 0x80] &= 0x0F
        return b

    assert np.array_equal(canon(got), canon(c.bytes))
    live = slots >= 0
    for odt, name in ((torch.float32, "fp32"), (torch.bfloat16, "bf16")):
        ko, vo = [torch.full((t, h, d), 5.0, dtype=odt, device="cuda") for _ in range(2)]
        df11.df11_kv4_gather(handle, sd.data_ptr(), t, ko.data_ptr(), vo.data_ptr(), dtype=name, err_ptr=err.data_ptr(),
                             stream=stream())
        torch.cuda.synchronize()
        for o, w in ((ko, c.k), (vo, c.v)):
            o = o.double().cpu().numpy()
            assert (o[~live] == 5.0).all()
            w = w[slots[live]]
            # one rounding to FP32 (of level * s * scale, the first product exact), then one to BF16
            tol = np.abs(w) * (2.0 ** -24 if name == "fp32" else 2.0 ** -24 + 2.0 ** -8 * (1 + 2.0 ** -24))
            assert (np.abs(o[live] - w) <= tol).all()
            if np.log2(gk) % 1 == 0 and np.log2(gv) % 1 == 0:
                assert np.array_equal(o[live], w)
    # one side only
    ko = torch.full((t, h, d), 5.0, dtype=torch.bfloat16, device="cuda")
    df11.df11_kv4_gather(handle, sd.data_ptr(), t, 0, ko.data_ptr(), stream=stream())
    assert torch.equal(ko, vo)
    assert err.item() == 0


def test_append_every_bf16_against_every_scale(df11):
    """All finite BF16 values beside block maxima of every mantissa, both signs: each level border is met exactly."""
    x = np.arange(1 << 16, dtype=np.uint32)
    x = (x << 16).view(np.float32)
    x = x[np.isfinite(x) & (np.abs(x) < 1e30) & (np.abs(x) > 1e-30)]
    g = np.random.default_rng(0)
    near = x[(np.abs(x) >= 2.0 ** -4) & (np.abs(x) < 32)]
    t, h, d = 512, 8, 64
    k = g.choice(near, (t, h, d))
    v = g.choice(x, (t, h, d))
    c = ref.Cache(t // 16, 16, h, d, 1.0, 1.0)
    handle, pages = device_cache(df11, c)
    kd, vd, sd = dev(k, torch.bfloat16), dev(v, torch.bfloat16), dev(np.arange(t), torch.int64)
    df11.df11_kv4_append(handle, kd.data_ptr(), h * d, vd.data_ptr(), h * d, sd.data_ptr(), t, stream=stream())
    ko, vo = [torch.zeros(t, h, d, device="cuda") for _ in range(2)]
    df11.df11_kv4_gather(handle, sd.data_ptr(), t, ko.data_ptr(), vo.data_ptr(), dtype="fp32", stream=stream())
    torch.cuda.synchronize()
    for o, y in ((ko, k), (vo, v)):
        assert np.array_equal(o.cpu().numpy().astype(np.float64), ref.quantize(y, 1.0)[2])


def test_append_non_finite_and_out_of_range(df11):
    c = ref.Cache(2, 16, 1, 64, 1.0, 1.0, fill=0x11)
    handle, pages = device_cache(df11, c)
    k = np.ones((4, 1, 64), np.float32)
    k[0, 0, 3] = np.inf
    k[1, 0, 20] = -np.inf
    k[2, 0, 40] = np.nan
    k[3] = np.nan
    slots = np.array([0, 5, 17, 31])
    kd, sd, err = dev(k, torch.float32), dev(slots, torch.int64), word()
    df11.df11_kv4_append(handle, kd.data_ptr(), 64, kd.data_ptr(), 64, sd.data_ptr(), 4, dtype="fp32",
                         err_ptr=err.data_ptr(), stream=stream())
    ko, vo = [torch.zeros(4, 1, 64, device="cuda") for _ in range(2)]
    df11.df11_kv4_gather(handle, sd.data_ptr(), 4, ko.data_ptr(), vo.data_ptr(), dtype="fp32", stream=stream())
    torch.cuda.synchronize()
    want = ref.quantize(k, 1.0)[2]
    assert err.item() == 0 and np.array_equal(ko.cpu().numpy(), want) and torch.equal(ko, vo)
    # slots past the cache: flagged, nothing written
    before = pages.clone()
    sd = dev([32, 1 << 40, -1, -(1 << 40)], torch.int64)
    df11.df11_kv4_append(handle, kd.data_ptr(), 64, kd.data_ptr(), 64, sd.data_ptr(), 4, dtype="fp32",
                         err_ptr=err.data_ptr(), stream=stream())
    torch.cuda.synchronize()
    assert err.item() == df11.DEV_ERR_PAGES and torch.equal(pages, before)
    err.zero_()
    ko.fill_(9.0)
    df11.df11_kv4_gather(handle, sd.data_ptr(), 4, ko.data_ptr(), 0, dtype="fp32", err_ptr=err.data_ptr(), stream=stream())
    torch.cuda.synchronize()
    assert err.item() == df11.DEV_ERR_PAGES and (ko == 9.0).all()


# ------------------------------------------------------------------ attention

class Problem:
    """Requests (q, kv) over a cache whose every other byte is 0xFF: NaN scales in the rest of the last pages and in
    the pages of nobody; block-table entries past a request's pages are out of range."""

    def __init__(self, df11, lens, hq, h, d, page, seed=0, gk=0.5, gv=0.25, qscale=0.7, tail=3, kv_scale=1.0):
        g = np.random.default_rng(seed)
        self.df11, self.lens, self.hq, self.h, self.d, self.page = df11, lens, hq, h, d, page
        counts = [-(-kv // page) for _, kv in lens]
        c = self.c = ref.Cache(sum(counts) + 2, page, h, d, gk, gv, fill=0xFF)
        ids = g.permutation(c.n_pages)
        self.width = max(max(counts), 1) + 1
        self.table = np.full((len(lens), self.width), 1 << 30)
        at, slots, total = 0, [], sum(kv for _, kv in lens)
        for r, (n, (_, kv)) in enumerate(zip(counts, lens)):
            self.table[r, :n] = ids[at:at + n]
            at += n
            slots += [int(self.table[r, p // page]) * page + p % page for p in range(kv)]
        k = g.standard_normal((total, h, d)).astype(np.float32) * kv_scale
        k[..., 3] *= 6
        v = g.standard_normal((total, h, d)).astype(np.float32) * 0.6
        self.slots = np.array(slots, np.int64)
        self.handle, self.pages = device_cache(df11, c)
        if total:  # written by the library (its bytes are tested above), read back for the reference
            kd, vd, sd = dev(k, torch.bfloat16), dev(v, torch.bfloat16), dev(self.slots, torch.int64)
            df11.df11_kv4_append(self.handle, kd.data_ptr(), h * d, vd.data_ptr(), h * d, sd.data_ptr(), total,
                                 stream=stream())
            ko, vo = [torch.zeros(total, h, d, device="cuda") for _ in range(2)]
            df11.df11_kv4_gather(self.handle, sd.data_ptr(), total, ko.data_ptr(), vo.data_ptr(), dtype="fp32",
                                 stream=stream())
            torch.cuda.synchronize()
            self.k, self.v = ko.double().cpu(), vo.double().cpu()
        else:
            self.k = self.v = torch.zeros(0, h, d, dtype=torch.float64)
        self.starts = np.concatenate([[0], np.cumsum([n for n, _ in lens])])
        self.t = int(self.starts[-1]) + tail
        self.q = dev(g.standard_normal((self.t, hq * d + 8)) * qscale, torch.bfloat16)
        self.max_q = max(n for n, _ in lens)

    def run(self, causal=True, window=0, scale=None, ws=None, err=None, max_q=None, table=None, lse=True, sync=True):
        df11, hq, d = self.df11, self.hq, self.d
        max_q = self.max_q if max_q is None else max_q
        o = torch.full((self.t, hq * d + 16), 7.0, dtype=torch.bfloat16, device="cuda")
        lo = torch.full((self.t, hq), 7.0, device="cuda")
        need = df11.df11_kv4_attention_workspace_bytes(self.handle, hq, len(self.lens), self.t, max_q)
        assert need > 0
        ws = torch.zeros(need + 64, dtype=torch.uint8, device="cuda") if ws is None else ws
        qs, kl = dev(self.starts, torch.int32), dev([kv for _, kv in self.lens], torch.int32)
        tb = dev(self.table if table is None else table, torch.int32)
        err = word() if err is None else err
        self.df11.df11_kv4_attention(self.handle, self.q.data_ptr(), hq * d + 8, o.data_ptr(), hq * d + 16, hq, qs.data_ptr(),
                                     kl.data_ptr(), tb.data_ptr(), len(self.lens), self.width, self.t, max_q,
                                     d ** -0.5 if scale is None else scale, ws.data_ptr(), need, causal=causal,
                                     window=window, lse_ptr=lo.data_ptr() if lse else None, err_ptr=err.data_ptr(),
                                     stream=stream())
        self.keep = (qs, kl, tb, ws)
        if sync:
            torch.cuda.synchronize()
        return o, lo, err

    def want(self, causal=True, window=0, scale=None, kv_of=None):
        out, at = [], 0
        for r, (n, kv) in enumerate(self.lens):
            q = self.q[self.starts[r]:self.starts[r] + n, :self.hq * self.d].double().cpu().reshape(n, self.hq, self.d)
            out.append(ref.attention(q, self.k[at:at + kv], self.v[at:at + kv], causal, window,
                                     self.d ** -0.5 if scale is None else scale))
            at += kv
        return out

    def check(self, o, lse, **kw):
        hq, d = self.hq, self.d
        end = int(self.starts[-1])
        assert (o[:, hq * d:] == 7.0).all() and (o[end:] == 7.0).all() and (lse[end:] == 7.0).all()
        og, lg = o[:, :hq * d].double().cpu().reshape(-1, hq, d), lse.double().cpu()
        for r, (wo, wl, wmag, smag, vmax) in enumerate(self.want(**kw)):
            s, n = int(self.starts[r]), self.lens[r][0]
            bo, bl = ref.attention_bounds(wo, wl, wmag, smag, vmax, self.lens[r][1], d)
            e = (og[s:s + n] - wo).abs()
            assert (e <= bo).all(), (r, self.lens[r], float((e - bo).max()), float(e.max()))
            inf = torch.isinf(wl)
            assert torch.equal(lg[s:s + n][inf], wl[inf]), r
            assert ((lg[s:s + n] - wl).abs()[~inf] <= bl[~inf]).all(), (r, self.lens[r])


HEADS = [(32, 8, 128), (4, 4, 64), (8, 1, 128), (3, 1, 64), (20, 2, 64), (7, 7, 128), (34, 2, 128)]


@pytest.mark.parametrize("hq,h,d", HEADS)
@pytest.mark.parametrize("page", [16, 32, 64, 128])
def test_single_tokens(df11, hq, h, d, page):
    """Decode steps: lengths of none, one, below, at and past the pages, long ones."""
    lens = [(1, kv) for kv in (1, 0, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 700, 1, 2049)]
    p = Problem(df11, lens, hq, h, d, page, seed=hq + page)
    o, lse, err = p.run()
    assert err.item() == 0
    p.check(o, lse)


@pytest.mark.parametrize("hq,h,d", [(32, 8, 128), (4, 4, 64), (6, 2, 128), (16, 1, 64)])
@pytest.mark.parametrize("window", [0, 1, 20, 300])
def test_few_tokens(df11, hq, h, d, window):
    """Drafted tokens: up to 8 rows a request, rows before the first key among them, with sliding windows."""
    lens = [(2, 2), (8, 900), (3, 1), (5, 0), (1, 333), (0, 50), (8, 8), (7, 64), (2, 1025)]
    p = Problem(df11, lens, hq, h, d, 16, seed=window)
    o, lse, err = p.run(window=window)
    assert err.item() == 0
    p.check(o, lse, window=window)


@pytest.mark.parametrize("hq,h,d", [(32, 8, 128), (4, 4, 64), (6, 2, 128), (16, 1, 64), (5, 5, 128)])
@pytest.mark.parametrize("causal,window", [(True, 0), (True, 100), (False, 0)])
def test_prompts(df11, hq, h, d, causal, window):
    """Prompt chunks beside single tokens: tiles with odd ends, rows that see nothing, contexts shorter and longer
    than the chunk."""
    lens = [(130, 130), (1, 500), (257, 700), (64, 64), (33, 1000), (100, 40), (0, 10), (3, 0), (1, 1), (129, 129)]
    p = Problem(df11, lens, hq, h, d, 32, seed=hq)
    o, lse, err = p.run(causal=causal, window=window)
    assert err.item() == 0
    p.check(o, lse, causal=causal, window=window)


@pytest.mark.parametrize("page", [16, 64, 128])
@pytest.mark.parametrize("d", [64, 128])
def test_one_prompt(df11, page, d):
    p = Problem(df11, [(1030, 1030)], 4, 2, d, page, seed=page)
    o, lse, err = p.run()
    assert err.item() == 0
    p.check(o, lse)


def test_cross_attention_lengths(df11):
    """Without the mask, queries and keys of any two lengths: an encoder's states."""
    lens = [(1, 1500), (200, 77), (5, 1), (300, 300), (40, 0), (17, 129)]
    p = Problem(df11, lens, 6, 6, 64, 64, seed=3)
    o, lse, err = p.run(causal=False)
    assert err.item() == 0
    p.check(o, lse, causal=False)


@pytest.mark.parametrize("n", [1, 4, 160])
def test_many_requests(df11, n):
    """More requests than SMs, short ones among long: the keys of one are shared out between CTAs, of others not."""
    g = np.random.default_rng(n)
    lens = [(int(g.integers(0, n + 1)) if n > 1 else 1, int(g.integers(0, 200))) for _ in range(300 if n < 100 else 30)]
    lens[7] = (n, 3000)
    lens[-1] = (n, 2500)
    p = Problem(df11, lens, 8, 2, 64, 16, seed=n)
    o, lse, err = p.run()
    assert err.item() == 0
    p.check(o, lse)


@pytest.mark.parametrize("hq,h,d,page", [(8, 8, 64, 16), (8, 4, 128, 64), (4, 4, 64, 128)])
def test_long_batches(df11, hq, h, d, page):
    """Shares of several long units, and of long beside very short ones: units that begin, end or lie in a warp's part
    of a share, and such that span warps and CTAs."""
    g = np.random.default_rng(page)
    lens = [(1, int(x)) for x in g.integers(800, 4200, 48)]
    lens[5:5] = [(1, 3), (1, 0), (1, 64), (1, 65)] * 3
    lens[40:40] = [(1, 1)] * 30
    p = Problem(df11, lens, hq, h, d, page, seed=page)
    o, lse, err = p.run()
    assert err.item() == 0
    p.check(o, lse)
    for _ in range(3):
        o2, lse2, err = p.run(ws=p.keep[-1])
        assert err.item() == 0 and torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("hq,h,d", [(24, 8, 64), (8, 8, 128)])
def test_units_of_a_chunk_each(df11, hq, h, d):
    """Every chunk ends a unit, whose columns are mostly empty: a stage's position is replaced right after the rows are
    stored.  Again and again on one workspace, with equal bits."""
    p = Problem(df11, [(1, 1 + (7 * r) % 64) for r in range(600)], hq, h, d, 64, seed=hq)
    o, lse, err = p.run()
    assert err.item() == 0
    p.check(o, lse)
    for _ in range(20):
        o2, lse2, _ = p.run(ws=p.keep[-1], err=err)
        assert torch.equal(o, o2) and torch.equal(lse, lse2) and err.item() == 0


@pytest.mark.parametrize("lens", [[(1, 20000)], [(1, 2100), (1, 2300), (1, 9000)]])
def test_units_that_many_ctas_join(df11, lens):
    """Every unit spans CTAs and every CTA has parts of up to two: which one arrives last differs, the bits do not."""
    p = Problem(df11, lens, 8, 2, 64, 16, seed=len(lens))
    o, lse, err = p.run()
    assert err.item() == 0
    p.check(o, lse)
    for _ in range(50):
        o2, lse2, _ = p.run(ws=p.keep[-1], err=err)
        assert torch.equal(o, o2) and torch.equal(lse, lse2) and err.item() == 0


@pytest.mark.parametrize("n", [1, 200])
def test_score_ranges(df11, n):
    """Scores far apart (one key takes all), tiny and huge queries and keys, a scale of 0 and a negative one."""
    for qscale, kv_scale, scale in ((30.0, 4.0, None), (1e-30, 1.0, 1e28), (1e30, 1.0, 1e-31), (1.0, 1.0, 0.0),
                                    (1.0, 1.0, -0.3), (0.0, 1.0, None)):
        p = Problem(df11, [(n, 700), (1, 90)], 4, 2, 128, 16, qscale=qscale, kv_scale=kv_scale)
        o, lse, err = p.run(scale=scale)
        assert err.item() == 0
        p.check(o, lse, scale=scale)


@pytest.mark.parametrize("hq,h,d", [(4, 1, 128), (4, 1, 64), (9, 3, 64), (16, 4, 128), (24, 8, 64), (7, 7, 128)])
@pytest.mark.parametrize("causal,window", [(True, 0), (True, 333), (True, 5), (False, 0)])
def test_prompts_over_long_contexts(df11, hq, h, d, causal, window):
    """Few rows against many keys, which several CTAs share: short last tiles, parts without a step, rows that see
    keys of one part only or none at all."""
    lens = [(90, 3000)] if h < 7 else [(90, 3000), (300, 1025)]
    for lens in (lens, [(257, 257)], [(200, 1300), (1, 800), (100, 30), (129, 385)], [(100, 0), (131, 2047)]):
        p = Problem(df11, lens, hq, h, d, 32, seed=hq)
        o, lse, err = p.run(causal=causal, window=window)
        assert err.item() == 0
        p.check(o, lse, causal=causal, window=window)
        o2, lse2, _ = p.run(causal=causal, window=window)
        assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("lens", [[(1, 900), (2, 300)], [(300, 300), (70, 2500)], [(1100, 1100)] * 3])
def test_nan_queries(df11, lens):
    """A NaN in a head's query makes that row NaN and leaves every other as it is."""
    p = Problem(df11, lens, 8, 4, 64, 16)
    o, lse, _ = p.run()
    rows = sorted({0, int(p.starts[1]) - 1, int(p.starts[-1]) - 1})
    for t in rows:
        p.q[t, 3 * 64 + 5] = float("nan")
    o2, lse2, err = p.run()
    assert err.item() == 0
    for t in rows:
        assert torch.isnan(o2[t, 192:256].float()).all() and torch.isnan(lse2[t, 3])
        o2[t, 192:256], lse2[t, 3] = o[t, 192:256], lse[t, 3]
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


def test_split_scales(df11):
    """Cache scales that are no powers of two."""
    p = Problem(df11, [(1, 1000), (70, 300)], 4, 2, 64, 32, gk=0.37, gv=1.9)
    o, lse, err = p.run()
    assert err.item() == 0
    p.check(o, lse)


@pytest.mark.parametrize("lens", [[(1, 3000)] * 3, [(150, 900), (1, 2000)]])
def test_repeats_bit_for_bit(df11, lens):
    """The same call on the same workspace, again and again and on another stream: equal bits; without lse too."""
    p = Problem(df11, lens, 8, 2, 128, 16)
    o, lse, err = p.run()
    ws = p.keep[-1]
    for _ in range(5):
        o2, lse2, _ = p.run(ws=ws, err=err)
        assert torch.equal(o, o2) and torch.equal(lse, lse2)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        o3, _, _ = p.run(ws=ws, err=err, lse=False)
    assert torch.equal(o, o3) and err.item() == 0


def test_two_calls_at_once(df11):
    """Two streams, a workspace each."""
    a, b = Problem(df11, [(1, 5000)] * 4, 8, 2, 128, 16, seed=1), Problem(df11, [(90, 900), (1, 7000)], 8, 2, 64, 32, seed=2)
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    outs = []
    for _ in range(3):
        with torch.cuda.stream(s):
            x = a.run(sync=False)
        with torch.cuda.stream(t):
            y = b.run(sync=False)
        torch.cuda.synchronize()
        outs.append((x, y))
    for x, y in outs:
        assert x[2].item() == 0 and y[2].item() == 0
        a.check(x[0], x[1])
        b.check(y[0], y[1])


def test_damaged_tables_are_flagged(df11):
    """Entries out of range: flagged, their keys left out, everything else as it was."""
    for n in (1, 140):
        p = Problem(df11, [(n, 400), (n, 300)], 4, 2, 64, 16)
        good, lse0, err = p.run()
        assert err.item() == 0
        table = p.table.copy()
        table[1, 3] = -1
        table[1, 5] = p.c.n_pages
        table[1, 18] = -(1 << 31)
        o, lse, err = p.run(table=table)
        assert err.item() == df11.DEV_ERR_PAGES
        rows = slice(0, n)
        assert torch.equal(o[rows], good[rows]) and torch.equal(lse[rows], lse0[rows])
        assert torch.isfinite(o[n:2 * n].float()).all()
        # as if those keys were not there (single tokens see every key: compare with the reference without them)
        if n == 1:
            drop = [j for j in range(300) if j // 16 in (3, 5, 18)]
            keep = [j for j in range(300) if j not in drop]
            q = p.q[1:2, :4 * 64].double().cpu().reshape(1, 4, 64)
            k, v = p.k[400:][keep], p.v[400:][keep]
            wo, wl, wm, sm, vm = ref.attention(q, k, v, True, 0, 0.125)
            bo, bl = ref.attention_bounds(wo, wl, wm, sm, vm, 300, 64)
            assert ((o[1:2, :256].double().cpu().reshape(1, 4, 64) - wo).abs() <= bo).all()
            assert ((lse[1:2].double().cpu() - wl).abs() <= bl).all()


def test_lengths_past_the_table_are_flagged(df11):
    for n in (1, 140):
        p = Problem(df11, [(n, 400), (n, 330)], 4, 2, 64, 16)
        good, _, _ = p.run()
        p.lens = [(n, 400), (n, 100000)]
        table = p.table.copy()
        table[1] = table[1, 0]
        o, lse, err = p.run(table=table)
        assert err.item() == df11.DEV_ERR_PAGES and torch.equal(o[:n], good[:n])
        assert torch.isfinite(o[n:2 * n].float()).all()
        p.lens = [(n, 400), (n, -3)]  # a negative length holds no key
        o, lse, err = p.run()
        assert torch.equal(o[:n], good[:n]) and (o[n:2 * n, :256] == 0).all() and torch.isneginf(lse[n:2 * n]).all()


def test_bad_row_starts_are_flagged(df11):
    p = Problem(df11, [(3, 40), (5, 60), (2, 30)], 4, 2, 64, 16)
    good, _, _ = p.run()
    # longer than max_q_len: not written
    o, _, err = p.run(max_q=4)
    assert err.item() == df11.DEV_ERR_AUX
    assert torch.equal(o[:3], good[:3]) and torch.equal(o[8:], good[8:]) and (o[3:8] == 7.0).all()
    # descending and past the rows
    starts = p.starts.copy()
    for bad in ([0, 8, 3, 10], [0, 3, 8, 100], [-4, 3, 8, 10]):
        p.starts = np.array(bad)
        o, _, err = p.run(max_q=200)
        assert err.item() == df11.DEV_ERR_AUX
        assert torch.isfinite(o.float()).all()
    p.starts = starts


def test_graph_replays_with_other_lengths(df11):
    """One captured call, replayed after the lengths, rows and tables on the device changed."""
    big = [(1, 1500), (1, 1500), (1, 1500)]
    p = Problem(df11, big, 8, 2, 128, 16, tail=0)
    o, lse = torch.empty(3, 8 * 128, dtype=torch.bfloat16, device="cuda"), torch.empty(3, 8, device="cuda")
    need = df11.df11_kv4_attention_workspace_bytes(p.handle, 8, 3, 3, 1)
    ws = torch.zeros(need, dtype=torch.uint8, device="cuda")
    qs, kl, tb = dev(p.starts, torch.int32), dev([1500] * 3, torch.int32), dev(p.table, torch.int32)
    q = p.q[:, :1024].contiguous()

    def call():
        df11.df11_kv4_attention(p.handle, q.data_ptr(), 1024, o.data_ptr(), 1024, 8, qs.data_ptr(), kl.data_ptr(),
                                tb.data_ptr(), 3, p.width, 3, 1, 128 ** -0.5, ws.data_ptr(), need, lse_ptr=lse.data_ptr(),
                                stream=stream())

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for lens in ([1500, 1500, 1500], [0, 1, 1499], [33, 700, 64], [1500, 2, 16]):
        kl.copy_(torch.tensor(lens, dtype=torch.int32))
        o.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        got = o.clone(), lse.clone()
        call()
        torch.cuda.synchronize()
        assert torch.equal(o, got[0]) and torch.equal(lse, got[1])
        for r, n in enumerate(lens):
            wo, wl, wm, sm, vm = ref.attention(q[r:r + 1].double().cpu().reshape(1, 8, 128), p.k[1500 * r:1500 * r + n],
                                               p.v[1500 * r:1500 * r + n], True, 0, 128 ** -0.5)
            bo, _ = ref.attention_bounds(wo, wl, wm, sm, vm, n, 128)
            assert ((got[0][r:r + 1].double().cpu().reshape(1, 8, 128) - wo).abs() <= bo).all()


@pytest.mark.parametrize("hq,h,d", [(128, 1, 64), (300, 1, 128), (130, 130, 64)])
def test_wide_groups_and_many_heads(df11, hq, h, d):
    """A single token's rows of one cache head past those of the few-row kernel, and more cache heads than SMs."""
    p = Problem(df11, [(1, 700), (1, 1), (2, 90), (1, 0)] if h == 1 else [(1, 90), (3, 40)], hq, h, d, 16, seed=hq)
    for window in (0, 33):
        o, lse, err = p.run(window=window)
        assert err.item() == 0
        p.check(o, lse, window=window)


@pytest.mark.parametrize("n", [2, 140])
def test_widest_bounds(df11, n):
    """The largest window and the largest bound on a request's rows change nothing."""
    p = Problem(df11, [(n, 500), (n, n), (n, 1)], 4, 2, 64, 16)
    o, lse, _ = p.run()
    for kw in (dict(window=2 ** 31 - 1), dict(max_q=2 ** 31 - 1)):
        o2, lse2, err = p.run(**kw)
        assert err.item() == 0
        p.check(o2, lse2)


@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31 - 3, 2 ** 30])
@pytest.mark.parametrize("hq,h,d", [(1, 1, 64), (2, 2, 128), (4, 1, 64)])
def test_wide_windows_of_more_rows_than_keys(df11, hq, h, d, window):
    """Rows at positions far below 0, whose distance to a wide window's start passes 32 bits: as without a window."""
    lens = [(30, 20), (8, 5), (8, 4), (24, 20), (7, 0), (16, 33)] if hq == h else [(8, 5), (8, 4), (7, 0), (8, 33), (16, 2)]
    p = Problem(df11, lens, hq, h, d, 16, seed=hq)
    o, lse, err = p.run(window=window)
    assert err.item() == 0
    p.check(o, lse)
    o2, lse2, _ = p.run()
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("n", [2, 140])
def test_rows_before_the_first_request(df11, n):
    """Row starts that begin past row 0: the rows before are left as they were."""
    p = Problem(df11, [(n, 500), (n, 300)], 4, 2, 64, 16, tail=5)
    p.starts = p.starts + 3
    o, lse, err = p.run()
    assert err.item() == 0 and (o[:3] == 7.0).all() and (lse[:3] == 7.0).all()
    p.check(o, lse)


def test_graph_replays_a_mixed_batch(df11):
    """Both kernels in one captured call, replayed with other lengths: rows go from one kernel to the other, requests
    lose all their rows or keys, and what follows in the graph reads what both have written."""
    lens = [(90, 1200), (4, 900), (40, 700), (1, 1300)]
    p = Problem(df11, lens, 8, 2, 64, 16, tail=0)
    t, hq, d = p.t, 8, 64
    q = p.q[:, :hq * d].contiguous()
    o, lse = torch.empty(t, hq * d, dtype=torch.bfloat16, device="cuda"), torch.empty(t, hq, device="cuda")
    need = df11.df11_kv4_attention_workspace_bytes(p.handle, hq, 4, t, 90)
    ws = torch.zeros(need, dtype=torch.uint8, device="cuda")
    qs, kl, tb, err = dev(p.starts, torch.int32), dev([kv for _, kv in lens], torch.int32), dev(p.table, torch.int32), word()

    def call():
        df11.df11_kv4_attention(p.handle, q.data_ptr(), hq * d, o.data_ptr(), hq * d, hq, qs.data_ptr(), kl.data_ptr(),
                                tb.data_ptr(), 4, p.width, t, 90, d ** -0.5, ws.data_ptr(), need, lse_ptr=lse.data_ptr(),
                                err_ptr=err.data_ptr(), stream=stream())
        return o.float() * 2

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        twice = call()
    for ns, kvs in (([90, 4, 40, 1], [1200, 900, 700, 1300]), ([4, 90, 1, 40], [1200, 900, 33, 1300]),
                    ([0, 0, 0, 0], [5, 5, 5, 5]), ([17, 16, 90, 12], [0, 16, 90, 1]), ([1, 2, 3, 4], [1200, 900, 700, 1300])):
        starts = np.concatenate([[0], np.cumsum(ns)])
        qs.copy_(torch.tensor(starts, dtype=torch.int32))
        kl.copy_(torch.tensor(kvs, dtype=torch.int32))
        o.fill_(7.0)
        lse.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(twice, o.float() * 2) and (o[starts[-1]:] == 7.0).all() and err.item() == 0
        at = 0
        for r, (n, kv) in enumerate(zip(ns, kvs)):
            rows = slice(int(starts[r]), int(starts[r + 1]))
            w = ref.attention(q[rows].double().cpu().reshape(n, hq, d), p.k[at:at + kv], p.v[at:at + kv], True, 0, d ** -0.5)
            at += lens[r][1]
            bo, _ = ref.attention_bounds(*w, kv, d)
            assert ((o[rows].double().cpu().reshape(n, hq, d) - w[0]).abs() <= bo).all(), (r, n, kv)


def test_more_prompts_than_are_sorted(df11):
    """600 requests, 130 of them with more rows than the few-row kernel takes."""
    g = np.random.default_rng(0)
    lens = [(int(g.integers(17, 40)) if r % 5 == 3 else int(g.integers(0, 3)), int(g.integers(0, 90))) for r in range(600)]
    lens[7] = (130, 500)
    for some in (lens, lens[:300]):  # in two rounds of the CTA's threads, and in one
        p = Problem(df11, some, 4, 1, 64, 16, seed=9)
        o, lse, err = p.run()
        assert err.item() == 0
        p.check(o, lse)


@pytest.mark.parametrize("n", [1, 100])
def test_no_pages(df11, n):
    """A table without columns: requests without keys are zeros, others flagged; with no error word as well."""
    p = Problem(df11, [(n, 0), (n, 0)], 4, 2, 64, 16)
    q, o = p.q, torch.full((2 * n, 256), 7.0, dtype=torch.bfloat16, device="cuda")
    need = df11.df11_kv4_attention_workspace_bytes(p.handle, 4, 2, 2 * n, n)
    ws = torch.zeros(need, dtype=torch.uint8, device="cuda")
    qs = dev([0, n, 2 * n], torch.int32)
    for kvs, want in (([0, 0], 0), ([0, 9], df11.DEV_ERR_PAGES)):
        for err in (word(), None):
            o.fill_(7.0)
            kl = dev(kvs, torch.int32)
            df11.df11_kv4_attention(p.handle, q.data_ptr(), q.shape[1], o.data_ptr(), 256, 4, qs.data_ptr(), kl.data_ptr(),
                                    0, 2, 0, 2 * n, n, 0.125, ws.data_ptr(), need,
                                    err_ptr=err.data_ptr() if err is not None else None, stream=stream())
            torch.cuda.synchronize()
            assert (o == 0).all() and (err is None or err.item() == want)


@pytest.mark.slow
def test_offsets_past_32_bits(df11):
    """A cache of 5 GB whose used pages lie at its end."""
    page, h, d = 64, 8, 128
    size = df11.df11_kv4_page_bytes(page, h, d)
    n_pages = 5 * 2 ** 30 // size
    pages = torch.full((n_pages * size,), 0xFF, dtype=torch.uint8, device="cuda")
    c = df11.Kv4Cache(pages.data_ptr(), n_pages, page, h, d, 1.0, 1.0)
    kv = 200
    ids = [n_pages - 1, 3, n_pages - 7, n_pages - 2]
    slots = dev([ids[j // page] * page + j % page for j in range(kv)], torch.int64)
    g = np.random.default_rng(0)
    k, v = [dev(g.standard_normal((kv, h, d)), torch.bfloat16) for _ in range(2)]
    df11.df11_kv4_append(c, k.data_ptr(), h * d, v.data_ptr(), h * d, slots.data_ptr(), kv, stream=stream())
    ko, vo = [torch.zeros(kv, h, d, device="cuda") for _ in range(2)]
    df11.df11_kv4_gather(c, slots.data_ptr(), kv, ko.data_ptr(), vo.data_ptr(), dtype="fp32", stream=stream())
    assert np.array_equal(ko.cpu().numpy(), ref.quantize(k.float().cpu().numpy(), 1.0)[2])
    table, kl = dev([ids], torch.int32), dev([kv], torch.int32)
    for n in (1, 150):
        q = dev(g.standard_normal((n, h * d)), torch.bfloat16)
        o, qs, err = torch.zeros_like(q), dev([0, n], torch.int32), word()
        need = df11.df11_kv4_attention_workspace_bytes(c, h, 1, n, n)
        ws = torch.zeros(need, dtype=torch.uint8, device="cuda")
        df11.df11_kv4_attention(c, q.data_ptr(), h * d, o.data_ptr(), h * d, h, qs.data_ptr(), kl.data_ptr(),
                                table.data_ptr(), 1, 4, n, n, d ** -0.5, ws.data_ptr(), need, err_ptr=err.data_ptr(),
                                stream=stream())
        torch.cuda.synchronize()
        wo, wl, wm, sm, vm = ref.attention(q.double().cpu().reshape(n, h, d), ko.double().cpu(), vo.double().cpu(), True, 0,
                                           d ** -0.5)
        bo, _ = ref.attention_bounds(wo, wl, wm, sm, vm, kv, d)
        assert err.item() == 0 and ((o.double().cpu().reshape(n, h, d) - wo).abs() <= bo).all()


# ------------------------------------------------------------------ one attention step of a compressed block

class Step:
    """x -> q, k, v (fused decode + GEMM) -> extend, norm + rotation, append, attention -> o -> y (fused GEMM)."""

    def __init__(self, df11, reqs=3, hq=8, h=2, d=64, page=16, seed=0):
        from entropy_decoding_b200 import synth
        g = np.random.default_rng(seed)
        self.df11, self.reqs, self.hq, self.h, self.d, self.page, self.hidden = df11, reqs, hq, h, d, page, 256
        self.shapes = [(256, hq * d), (256, h * d), (256, h * d), (hq * d, 256)]
        bits = [synth.to_bf16_bits((g.standard_normal(k * n) / np.sqrt(k)).astype(np.float32)) for k, n in self.shapes]
        tiled = [df11.df11_gemm_tile_weights(b, k, n) for b, (k, n) in zip(bits, self.shapes)]
        cb = df11.df11_build_codebook("bf16", tiled)
        self.blobs = [df11.df11_encode(cb, t) for t in tiled]
        for b in self.blobs:
            df11.upload(b)
        self.w = [(b.astype(np.uint32) << 16).view(np.float32).reshape(s).astype(np.float64)
                  for b, s in zip(bits, self.shapes)]
        self.width, self.n_pages, self.t = 8, 40, 12  # room for 12 rows a step
        i32 = dict(dtype=torch.int32, device="cuda")
        self.pages = torch.full((self.n_pages, df11.df11_kv4_page_bytes(page, h, d)), 0xFF, dtype=torch.uint8, device="cuda")
        self.cache = df11.Kv4Cache(self.pages.data_ptr(), self.n_pages, page, h, d, 0.5, 0.25)
        self.free, self.n_free = torch.arange(self.n_pages, **i32), torch.tensor([self.n_pages], **i32)
        self.table = torch.full((reqs, self.width), -1, **i32)
        self.kv, self.new = torch.zeros(reqs, **i32), torch.zeros(reqs, **i32)
        self.kv_out, self.q_start, self.n_free_out = torch.zeros(reqs, **i32), torch.zeros(reqs + 1, **i32), torch.zeros(1, **i32)
        self.slots, self.pos = torch.zeros(self.t, dtype=torch.int64, device="cuda"), torch.zeros(self.t, **i32)
        self.x = torch.zeros(self.t, 256, dtype=torch.bfloat16, device="cuda")
        f32 = dict(dtype=torch.float32, device="cuda")
        self.q, self.k, self.v = [torch.zeros(self.t, n, **f32) for _, n in self.shapes[:3]]
        self.y = torch.zeros(self.t, 256, **f32)
        bf = dict(dtype=torch.bfloat16, device="cuda")
        self.qr, self.kr, self.o = torch.zeros(self.t, hq * d, **bf), torch.zeros(self.t, h * d, **bf), torch.zeros(self.t, hq * d, **bf)
        self.wq, self.wk = [dev(1 + 0.2 * g.standard_normal(d), torch.bfloat16) for _ in range(2)]
        self.freq = dev(10000.0 ** (-np.arange(0, d, 2) / d), torch.float64)
        need = df11.df11_kv4_attention_workspace_bytes(self.cache, hq, reqs, self.t, self.t)
        self.ws = torch.zeros(need, dtype=torch.uint8, device="cuda")
        self.err = word()

    def step(self):
        f, s, e = self.df11, stream(), self.err.data_ptr()
        d, hq, h, t = self.d, self.hq, self.h, self.t
        f.df11_kv_extend(self.kv.data_ptr(), self.new.data_ptr(), self.reqs, self.free.data_ptr(), self.n_free.data_ptr(),
                         self.table.data_ptr(), self.width, self.page, self.kv_out.data_ptr(), self.q_start.data_ptr(),
                         self.slots.data_ptr(), self.pos.data_ptr(), t, self.n_free_out.data_ptr(), e, s)
        for y in (self.q, self.k, self.v, self.y):
            y.zero_()
        f.df11_decode_gemm([(b, *sh, self.x.data_ptr(), y.data_ptr())
                            for b, sh, y in zip(self.blobs[:3], self.shapes, (self.q, self.k, self.v))], t, e, s)
        f.df11_qk_norm_rope((self.q.data_ptr(), hq * d, self.wq.data_ptr(), self.qr.data_ptr(), hq * d, hq),
                            (self.k.data_ptr(), h * d, self.wk.data_ptr(), self.kr.data_ptr(), h * d, h), t, d,
                            self.pos.data_ptr(), self.freq.data_ptr(), d, stream=s)
        # the rotated keys are BF16, the values FP32 from the GEMM: one type a call
        vb = self.v.to(torch.bfloat16)
        self.vb = vb
        f.df11_kv4_append(self.cache, self.kr.data_ptr(), h * d, vb.data_ptr(), h * d, self.slots.data_ptr(), t, err_ptr=e,
                          stream=s)
        f.df11_kv4_attention(self.cache, self.qr.data_ptr(), hq * d, self.o.data_ptr(), hq * d, hq, self.q_start.data_ptr(),
                             self.kv_out.data_ptr(), self.table.data_ptr(), self.reqs, self.width, t, t, d ** -0.5,
                             self.ws.data_ptr(), self.ws.numel(), err_ptr=e, stream=s)
        f.df11_decode_gemm([(self.blobs[3], *self.shapes[3], self.o.data_ptr(), self.y.data_ptr())], t, e, s)
        self.kv.copy_(self.kv_out)
        self.n_free.copy_(self.n_free_out)


@pytest.mark.parametrize("captured", [False, True])
def test_attention_step_of_a_compressed_block(df11, captured):
    """Prompts, then single tokens, then drafted ones, padded to 12 rows, each stage against the 64-bit form of its own
    inputs; the same with the whole step captured once and replayed."""
    s = Step(df11)
    graph = None
    if captured:
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            s.step()  # no new tokens: changes nothing
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            s.step()
    g = np.random.default_rng(9)
    hist = [([], []) for _ in range(s.reqs)]
    kv = [0] * s.reqs
    w64 = [w for w in s.w]
    for new in ([5, 7, 0], [5, 1, 4], [1, 1, 1], [0, 3, 2], [1, 0, 1]):
        s.o.fill_(0.0)
        s.x.copy_(dev(g.standard_normal((s.t, 256)), torch.bfloat16))
        s.new.copy_(torch.tensor(new, dtype=torch.int32))
        graph.replay() if captured else s.step()
        torch.cuda.synchronize()
        assert s.err.item() == 0
        rows = sum(new)
        x = s.x.double().cpu().numpy()
        for y, w in ((s.q, w64[0]), (s.k, w64[1]), (s.v, w64[2])):
            bound = (256 + 16) * 2.0 ** -24 * (np.abs(x) @ np.abs(w))
            assert (np.abs(y.double().cpu().numpy() - x @ w) <= bound).all()
        pos = s.pos.cpu().numpy()
        freq = s.freq.cpu().numpy()
        for y, o, w, heads in ((s.q, s.qr, s.wq, s.hq), (s.k, s.kr, s.wk, s.h)):
            want, mag = ref.norm_rope(y.double().cpu().numpy().reshape(s.t, heads, s.d), w.double().cpu().numpy(), pos, freq,
                                      s.d, False, 1e-6)
            e = mag * ((s.d / 2 + 8) * 2.0 ** -24 + 2.0 ** -21)
            assert (np.abs(o.double().cpu().numpy().reshape(want.shape) - want) <= e + 2.0 ** -8 * (np.abs(want) + e)).all()
        kq = ref.quantize(s.kr.float().cpu().numpy().reshape(s.t, s.h, s.d), 0.5)[2]
        vq = ref.quantize(s.v.cpu().numpy().reshape(s.t, s.h, s.d), 0.25)[2]
        at = 0
        q64, o64 = s.qr.double().cpu().reshape(s.t, s.hq, s.d), s.o.double().cpu().reshape(s.t, s.hq, s.d)
        for r, n in enumerate(new):
            hist[r][0].extend(kq[at:at + n])
            hist[r][1].extend(vq[at:at + n])
            kv[r] += n
            if n:
                k, v = torch.tensor(np.array(hist[r][0])), torch.tensor(np.array(hist[r][1]))
                wo, wl, wm, sm, vm = ref.attention(q64[at:at + n], k, v, True, 0, s.d ** -0.5)
                bo, _ = ref.attention_bounds(wo, wl, wm, sm, vm, kv[r], s.d)
                assert ((o64[at:at + n] - wo).abs() <= bo).all()
            at += n
        assert s.kv.cpu().tolist() == kv and (s.o[rows:] == 0).all()
        o = s.o.double().cpu().numpy()
        bound = (s.shapes[3][0] + 16) * 2.0 ** -24 * (np.abs(o) @ np.abs(w64[3]))
        assert (np.abs(s.y.double().cpu().numpy() - o @ w64[3]) <= bound).all()
