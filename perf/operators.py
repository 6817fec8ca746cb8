"""The paged int8 cache: appending keys and values to it, reading rows back, and attention over it.

A case is a dict; ``op`` says which operator a pass goes through:

  append   cache_append of the case's new rows, then cache_read of every page that it touched
  read     cache_read of whole sequences (the bf16 rows that routing and the routed forward take)
  forward  cache_forward of the case's query rows over the cached rows

Sizes: B sequences, H query heads over kv K/V heads of size d; ``len`` cached rows of the longest sequence (of the
append: rows held before it), ``rows`` new or query rows of the longest sequence; ``ragged`` in percent: how far
the shortest sequence lies below the longest; ``pad`` rows behind the last sequence that belong to none.
"""
import math
import random

import torch

own = False

PAGE = 64
PENALTY = (2.0, 0.20, 0.25, 6.0)
FRAME_S = 4.0 / 24.0  # seconds between latent frames


def _case(name, op, B, H, kv, d, length, rows, **more):
    c = {"name": name, "op": op, "B": B, "H": H, "kv": kv, "d": d, "len": length, "rows": rows, "ragged": 0, "pad": 0,
         "causal": False, "pen": False, "rope": "none"}
    c.update(more)
    return c


def listed():
    return [
        # one new token of each of eight running sequences, in the middle of a page: launch latency
        _case("append token B=8", "append", 8, 8, 8, 128, 1000, 1, ragged=60, rope="half"),
        # chunks of a ragged batch that begin and end inside pages, heads of 64, interleaved rotation
        _case("append ragged d=64", "append", 3, 24, 24, 64, 777, 1978, ragged=70, rope="interleaved", pad=37),
        # the 16,384 rows of a short clip, all 56 heads, into an empty cache
        _case("append clip H=56", "append", 1, 56, 56, 128, 0, 16384, rope="half"),
        # the conditioning rows (text, references, audio) of a long clip back as bf16
        _case("read prefix H=56", "read", 1, 56, 56, 128, 2079, 2079),
        # the cached rows of a ragged batch back as bf16
        _case("read ragged", "read", 5, 8, 8, 128, 16384, 16384, ragged=50),
        # one token over the conditioning rows, 56 heads of their own: the latency end
        _case("one row over 2,079", "forward", 1, 56, 56, 128, 2079, 1),
        # one token of each of 32 ragged sequences, grouped heads: the usual serving step
        _case("one row, B=32 ragged", "forward", 32, 32, 8, 128, 8192, 1, ragged=95, causal=True),
        # one token over the longest packed sequence, seven query heads on each K/V head
        _case("one row over 116,883", "forward", 1, 56, 8, 128, 116883, 1),
        # a few rows of each sequence (drafts being checked), heads of 64
        _case("five rows d=64", "forward", 6, 16, 4, 64, 3001, 5, ragged=40, causal=True, pad=3),
        # one latent frame of output rows over the cached guide clip, with the temporal penalty
        _case("frame over guide, penalty", "forward", 1, 8, 8, 128, 57402, 2126, pen=True),
        # a new chunk that attends itself and all rows before it
        _case("causal chunk B=4", "forward", 4, 16, 4, 128, 6000, 2500, ragged=45, causal=True),
        # a handful of audio or text rows over a long cache: between the token and the chunk
        _case("seventy rows over 16,384", "forward", 2, 16, 16, 128, 16384, 70),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("append", "append", "read", "forward", "forward", "forward", "forward"))
    while True:
        d = rng.choice((64, 128, 128))
        kv = rng.choice((1, 2, 4, 8, 8, 16, 56))
        g = rng.choice((1, 1, 2, 4, 5, 7, 8)) if kv < 56 else 1
        B = _log(rng, 1, 40)
        ragged = rng.choice((0, 30, 60, 95))
        pad = rng.choice((0, 0, 1, 29))
        if op == "forward":
            length = _log(rng, 1, 116883)
            rows = rng.choice((1, 1, _log(rng, 2, 8), _log(rng, 9, 200), _log(rng, 200, 2500)))
            causal, pen = rng.random() < 0.4, rng.random() < 0.25
            c = _case("", op, B, kv * g, kv, d, length, rows, ragged=ragged, pad=pad, causal=causal, pen=pen)
        elif op == "append":
            rope = rng.choice(("none", "half", "interleaved"))
            c = _case("", op, B, kv, kv, d, rng.choice((0, _log(rng, 1, 20000))), rng.choice((1, _log(rng, 1, 16384))),
                      ragged=ragged, pad=pad, rope=rope)
        else:
            length = _log(rng, 1, 16384)
            c = _case("", op, B, kv, kv, d, length, length, ragged=ragged, pad=pad)
        del c["name"]
        w = work(c)
        held = 2 * c["kv"] * c["B"] * (c["len"] + c["rows"]) * c["d"]
        scores = c["B"] * c["H"] * c["rows"] * c["len"] if op == "forward" else 0
        if w["bytes"] <= 7.0e8 and w["flops"] <= 4.9e11 and held <= 6.0e8 and scores <= 1.0e9:
            return c


def _lengths(case):
    """(cached rows, rows of the call) of each sequence."""
    B, out = case["B"], []
    for b in range(B):
        f = 1.0 - case["ragged"] / 100.0 * ((b * 7 + 3) % B) / max(1, B - 1) if B > 1 else 1.0
        n = max(1, int(round(case["rows"] * f))) if case["rows"] > 1 else case["rows"]
        length = int(round(case["len"] * f)) if case["len"] else 0
        if case["op"] == "read":
            n = length
        out.append((length, n))
    return out


def work(case):
    H, kv, d = case["H"], case["kv"], case["d"]
    by, fl = 0.0, 0.0
    for length, n in _lengths(case):
        if case["op"] == "append":
            table = 0 if case["rope"] == "none" else n * d * 4
            touched = length % PAGE + n  # rows read back, earlier rows of the first page included
            by += 2 * kv * n * d * 2 + table + 2 * kv * n * d + 2 * kv * touched * d * 2
            by += 8 * kv * (-(-touched // PAGE))
        elif case["op"] == "read":
            by += 2 * kv * n * d * 3 + 8 * kv * (-(-n // PAGE))
        else:
            seen = sum(max(0, length - n + i + 1) for i in range(n)) if case["causal"] else n * length
            by += 2 * kv * length * d + 8 * kv * (-(-length // PAGE)) + H * n * d * 4 + H * n * 4
            by += length * 4 + n * 4 if case["pen"] else 0
            fl += 4.0 * H * seen * d
    return {"bytes": float(by), "flops": fl}


def _inputs(case, seed):
    """Everything that the operators take, as plain tensors."""
    dev = "cuda"
    gen = torch.Generator(device=dev).manual_seed(seed)
    B, H, kv, d = case["B"], case["H"], case["kv"], case["d"]
    lens = _lengths(case)
    held = [length + (n if case["op"] == "append" else 0) for length, n in lens]
    pages = [-(-h // PAGE) for h in held]
    width = max(1, max(pages)) + 1
    total = sum(pages) + 3
    ids = torch.randperm(total, generator=gen, device=dev).to(torch.int32)
    table = torch.full((B, width), 0, dtype=torch.int32, device=dev)
    at = 0
    for b, n in enumerate(pages):
        table[b, :n] = ids[at:at + n]
        at += n
    s = {"case": case}
    for t in ("k", "v"):
        codes = torch.empty(total, kv, PAGE, d, dtype=torch.int8, device=dev)
        scale = torch.empty(total, kv, device=dev)
        step = max(1, (1 << 28) // (kv * PAGE * d))
        for p in range(0, total, step):  # rows with a mean of their own in every block, as in a frame of video
            x = torch.randn(min(step, total - p), kv, PAGE, d, generator=gen, device=dev)
            if t == "k":
                m = torch.randn(x.shape[0], kv, 1, d, generator=gen, device=dev)
                x += 2.0 * m / m.norm(dim=-1, keepdim=True)
            sc = x.abs().amax(dim=(2, 3)) / 127.0
            codes[p:p + step] = torch.round(x / sc[:, :, None, None]).clamp_(-127, 127).to(torch.int8)
            scale[p:p + step] = sc
        s[t + "_codes"], s[t + "_scale"] = codes, scale
    n_rows = [n for _, n in lens]
    T = sum(n_rows) + case["pad"]
    starts = [0]
    for n in n_rows:
        starts.append(starts[-1] + n)
    s["row_start"] = torch.tensor(starts, dtype=torch.int32, device=dev)
    s["length"] = torch.tensor([length for length, _ in lens], dtype=torch.int32, device=dev)
    s["table"] = table
    s["max_rows"] = max(n_rows)
    s["times"] = None
    if case["op"] == "append":
        s["k_new"] = torch.randn(kv, T, d, generator=gen, device=dev).to(torch.bfloat16)
        s["v_new"] = torch.randn(kv, T, d, generator=gen, device=dev).to(torch.bfloat16)
        if case["rope"] != "none":
            pos = torch.arange(max(held) + 1, device=dev, dtype=torch.float64)
            freq = 10000.0 ** (-torch.arange(d // 2, device=dev, dtype=torch.float64) * 2.0 / d)
            s["cos"] = torch.cos(pos[:, None] * freq).float()
            s["sin"] = torch.sin(pos[:, None] * freq).float()
        # what is read back: every page that the append touches, from its first row
        first = [length // PAGE * PAGE for length, _ in lens]
        back = [0]
        for (length, n), f in zip(lens, first):
            back.append(back[-1] + length + n - f)
        s["back_start"] = torch.tensor(back, dtype=torch.int32, device=dev)
        s["back_first"] = torch.tensor(first, dtype=torch.int32, device=dev)
        s["back_rows"] = back[-1]
    elif case["op"] == "read":
        s["back_start"], s["back_first"], s["back_rows"] = s["row_start"], torch.zeros_like(s["length"]), T
    else:
        s["q"] = torch.randn(H, T, d, generator=gen, device=dev).to(torch.bfloat16)
        s["out"] = torch.zeros(H, T, d, dtype=torch.bfloat16, device=dev)
        s["lse"] = torch.zeros(H, T, device=dev)
        s["q_times"] = None
        if case["pen"]:
            frame = max(1, case["rows"])  # cached rows: frame after frame of guide video, every 16th page none
            t = torch.arange(total * PAGE, device=dev) % 57402
            s["times"] = ((t // frame).float() * FRAME_S).view(total, PAGE).contiguous()
            s["times"][::16] = float("nan")
            s["q_times"] = (torch.randint(0, 27, (T,), generator=gen, device=dev).float() * FRAME_S)
            s["q_times"][::11] = float("nan")  # rows that are no output rows
    if "back_rows" in s:
        s["k_back"] = torch.zeros(kv, s["back_rows"], d, dtype=torch.bfloat16, device=dev)
        s["v_back"] = torch.zeros(kv, s["back_rows"], d, dtype=torch.bfloat16, device=dev)
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if own:
        import biased_attention_video_b200 as h3

        s["cache"] = h3.Cache(s["k_codes"], s["v_codes"], s["k_scale"], s["v_scale"], s["times"])
        s["rope"] = h3.Rope(s["cos"], s["sin"], interleaved=case["rope"] == "interleaved") if "cos" in s else None
        T = s["back_rows"] if "back_rows" in s else s["q"].shape[1]
        s["ws"] = h3.cache_workspace(s["cache"], case["H"], T, case["B"])
    return s


def run(s):
    op = s["case"]["op"]
    if own:
        import biased_attention_video_b200 as h3

        c = s["cache"]
        if op == "forward":
            o, lse = h3.cache_forward(c, s["q"], s["row_start"], s["length"], s["table"], causal=s["case"]["causal"],
                                      pen=PENALTY if s["case"]["pen"] else None, q_times=s["q_times"],
                                      max_rows=s["max_rows"], ws=s["ws"], out=s["out"], lse=s["lse"])
            return {"o": o, "lse": lse}
        if op == "append":
            h3.cache_append(c, s["k_new"], s["v_new"], s["row_start"], s["length"], s["table"], rope=s["rope"],
                            ws=s["ws"])
        k, v = h3.cache_read(c, s["back_start"], s["back_first"], s["table"], k_out=s["k_back"], v_out=s["v_back"],
                             ws=s["ws"])
    else:
        if op == "forward":
            return _plain_forward(s)
        if op == "append":
            _plain_append(s)
        k, v = _plain_read(s)
    return {"k": k, "v": v} if op == "read" else {"k": k, "v": v, "k_scale": s["k_scale"], "v_scale": s["v_scale"]}


# ---------------------------------------------------------------- plain forms


def _places(s, start, first, n):
    """(page, offset, sequence, position) of n packed rows; rows [start[b], start[b+1]) are positions from first[b]."""
    r = torch.arange(n, device=start.device)
    b = torch.searchsorted(start[1:].long(), r, right=True)
    pos = first.long()[b] + r - start.long()[b]
    return s["table"].long()[b, pos // PAGE], pos % PAGE, b, pos


def _rotate(s, x, pos):
    c, sn = s["cos"][pos], s["sin"][pos]
    half = x.shape[-1] // 2
    if s["case"]["rope"] == "half":
        a, b = x[..., :half], x[..., half:]
        return torch.cat((a * c - b * sn, b * c + a * sn), dim=-1)
    a, b = x[..., 0::2], x[..., 1::2]
    return torch.stack((a * c - b * sn, b * c + a * sn), dim=-1).flatten(-2)


def _plain_append(s):
    n = s["k_new"].shape[1] - s["case"]["pad"]
    page, off, b, pos = _places(s, s["row_start"], s["length"], n)
    held = torch.zeros(s["k_scale"].shape[0], dtype=torch.long, device=page.device)
    # rows that a touched page held before: the first new row's offset where the sequence stood in that page
    stood = s["length"].long()[b]
    held[page] = torch.where(pos // PAGE == stood // PAGE, stood % PAGE, 0)
    touched = torch.zeros_like(held, dtype=torch.bool)
    touched[page] = True
    c127 = torch.full((), 127.0, device=page.device)
    for t in ("k", "v"):
        x = s[t + "_new"][:, :n].float()
        if t == "k" and s["case"]["rope"] != "none":
            x = _rotate(s, x, pos)
        rows = x.abs().amax(dim=-1).t().contiguous()  # [n][heads]
        codes, scale = s[t + "_codes"], s[t + "_scale"]
        a = torch.zeros_like(scale).scatter_reduce_(0, page[:, None].expand_as(rows), rows, "amax") / c127
        old = torch.where(held[:, None] > 0, scale, 0.0)
        new = torch.maximum(torch.maximum(old, a), torch.full_like(a, 2.0 ** -100))
        new = torch.where(touched[:, None], new, scale)
        grown = torch.nonzero(touched & (held > 0))[:, 0]
        ratio = (old[grown] / new[grown])[:, :, None, None]
        codes[grown] = torch.round(codes[grown].float() * ratio).to(torch.int8)
        inv = torch.reciprocal(new)[page]
        codes[page, :, off] = torch.round(x.transpose(0, 1) * inv[:, :, None]).clamp_(-127, 127).to(torch.int8)
        scale.copy_(new)


def _plain_read(s):
    n = s["back_rows"] - (s["case"]["pad"] if s["case"]["op"] == "read" else 0)
    page, off, _, _ = _places(s, s["back_start"], s["back_first"], n)
    for t in ("k", "v"):
        x = s[t + "_codes"][page, :, off].float() * s[t + "_scale"][page][:, :, None]
        s[t + "_back"][:, :n] = x.transpose(0, 1).to(torch.bfloat16)
    return s["k_back"], s["v_back"]


def _plain_forward(s):
    case = s["case"]
    B, H, kv, d = case["B"], case["H"], case["kv"], case["d"]
    start, length, N = s["row_start"].long(), s["length"].long(), s["max_rows"]
    P = max(1, -(-case["len"] // PAGE))
    pages = s["table"][:, :P].long()

    def dequant(t):
        x = s[t + "_codes"][pages].float() * s[t + "_scale"][pages][..., None, None]
        return x.permute(0, 2, 1, 3, 4).reshape(B, kv, P * PAGE, d)

    n = start[1:] - start[:-1]
    i = torch.arange(N, device=start.device)
    j = torch.arange(P * PAGE, device=start.device)
    row = (start[:-1, None] + i).clamp(max=s["q"].shape[1] - 1)
    q = s["q"][:, row].float().view(kv, H // kv, B, N, d).permute(2, 0, 1, 3, 4).reshape(B, kv, H // kv * N, d)
    x = (q @ dequant("k").transpose(-1, -2)).view(B, kv, H // kv, N, P * PAGE)
    x *= 1.0 / math.sqrt(d)
    if case["pen"]:
        strength, window, falloff, cap = PENALTY
        dt = (s["q_times"][row][:, :, None] - s["times"][pages].reshape(B, 1, P * PAGE)).abs()
        pen = (strength * ((dt - window).clamp(min=0.0) / falloff) ** 2).clamp(max=cap)
        x -= torch.where(torch.isnan(dt), 0.0, pen)[:, None, None]
    seen = length[:, None]
    if case["causal"]:
        seen = length[:, None] - n[:, None] + i + 1
    x.masked_fill_((j >= seen.expand(B, N)[:, :, None])[:, None, None], -math.inf)
    m = x.amax(dim=-1, keepdim=True)
    m = torch.where(torch.isinf(m), 0.0, m)
    x -= m
    x.exp_()
    total = x.sum(dim=-1, keepdim=True)
    o = (x.view(B, kv, H // kv * N, P * PAGE) @ dequant("v")).view(B, kv, H // kv, N, d)
    o = o / torch.where(total > 0, total, 1.0)
    lse = (m + torch.log(total))[..., 0]
    valid = i < n[:, None]
    rows = row[valid]
    s["out"][:, rows] = o.permute(1, 2, 0, 3, 4).reshape(H, B, N, d)[:, valid].to(torch.bfloat16)
    s["lse"][:, rows] = lse.permute(1, 2, 0, 3).reshape(H, B, N)[:, valid]
    return {"o": s["out"], "lse": s["lse"]}


# ------------------------------------------------- the definition in 64 bits


def exact(case, seed):
    s = _inputs(case, seed)
    f64 = torch.float64
    lens, table = _lengths(case), s["table"].tolist()
    if case["op"] == "forward":
        return _exact_forward(case, s, lens, table)
    val = {t: s[t + "_codes"].to(f64) * s[t + "_scale"].to(f64)[:, :, None, None] for t in ("k", "v")}
    scale = {t: s[t + "_scale"].to(f64) for t in ("k", "v")}
    if case["op"] == "append":
        at = 0
        for b, (length, n) in enumerate(lens):
            for p0 in range(length // PAGE, (length + n - 1) // PAGE + 1):
                g = table[b][p0]
                lo, hi = max(length, p0 * PAGE), min(length + n, (p0 + 1) * PAGE)
                held = lo - p0 * PAGE if lo == length else 0
                for t in ("k", "v"):
                    x = s[t + "_new"][:, at + lo - length:at + hi - length].to(f64)
                    if t == "k" and case["rope"] != "none":
                        x = _turned(case, s, x, lo, hi)
                    old = scale[t][g].clone() if held else torch.zeros_like(scale[t][g])
                    new = torch.maximum(x.abs().amax(dim=(1, 2)) / 127.0, old).clamp(min=2.0 ** -100)
                    new = new.float().to(f64)  # a scale is stored in 32 bits
                    if held:
                        v = torch.round(val[t][g][:, :held] / new[:, None, None])
                        val[t][g][:, :held] = v * new[:, None, None]
                    q = torch.round(x / new[:, None, None]).clamp(-127, 127)
                    val[t][g][:, held:held + hi - lo] = q * new[:, None, None]
                    scale[t][g] = new
            at += n
    first, back = s["back_first"].tolist(), s["back_start"].tolist()
    out = {}
    for t in ("k", "v"):
        y = torch.zeros(case["kv"], s["back_rows"], case["d"], dtype=f64, device="cuda")
        for b in range(case["B"]):
            n = back[b + 1] - back[b]
            p = torch.arange(first[b], first[b] + n, device="cuda")
            g = s["table"][b].long()[p // PAGE]
            y[:, back[b]:back[b + 1]] = val[t][g, :, p % PAGE].transpose(0, 1)
        out[t] = y
    if case["op"] == "append":
        out["k_scale"], out["v_scale"] = scale["k"], scale["v"]
    return out


def _turned(case, s, x, lo, hi):
    """Rows at positions [lo, hi) as complex numbers times the unit numbers of their angles."""
    half = case["d"] // 2
    unit = torch.complex(s["cos"][lo:hi].double(), s["sin"][lo:hi].double())
    if case["rope"] == "half":
        z = torch.complex(x[..., :half].contiguous(), x[..., half:].contiguous()) * unit
        return torch.cat((z.real, z.imag), dim=-1)
    z = torch.view_as_complex(x.reshape(*x.shape[:-1], half, 2).contiguous()) * unit
    return torch.view_as_real(z).reshape(x.shape)


def _exact_forward(case, s, lens, table):
    f64 = torch.float64
    H, kv, d = case["H"], case["kv"], case["d"]
    o = torch.zeros(s["out"].shape, dtype=f64, device="cuda")
    lse = torch.zeros(s["lse"].shape, dtype=f64, device="cuda")
    at = 0
    for b, (length, n) in enumerate(lens):
        g = torch.tensor(table[b][:-(-length // PAGE)], dtype=torch.long, device="cuda")
        bias = torch.zeros(n, length, dtype=f64, device="cuda")
        if case["pen"] and length:
            tk = s["times"][g].reshape(-1)[:length].to(f64)
            dt = (s["q_times"][at:at + n].to(f64)[:, None] - tk).abs()
            strength, window, falloff, cap = PENALTY
            over = (torch.nan_to_num(dt, nan=0.0) - window).clamp(min=0.0) / falloff
            bias -= (strength * over * over).clamp(max=cap)
        if case["causal"]:
            hide = torch.arange(length, device="cuda") > length - n + torch.arange(n, device="cuda")[:, None]
            bias.masked_fill_(hide, -math.inf)
        for h in range(H):
            k = (s["k_codes"][g, h * kv // H].to(f64) * s["k_scale"][g, h * kv // H].to(f64)[:, None, None])
            v = (s["v_codes"][g, h * kv // H].to(f64) * s["v_scale"][g, h * kv // H].to(f64)[:, None, None])
            k, v = k.reshape(-1, d)[:length], v.reshape(-1, d)[:length]
            x = s["q"][h, at:at + n].to(f64) @ k.t() / math.sqrt(d) + bias
            y = torch.logsumexp(x, dim=-1)
            lse[h, at:at + n] = y
            w = torch.exp(x - torch.where(torch.isinf(y), 0.0, y)[:, None])
            o[h, at:at + n] = w @ v
        at += n
    return {"o": o, "lse": lse}


if __name__ == "__main__":
    for c in listed() + [draw(random.Random(i)) for i in range(6)]:
        print(c.get("name", "drawn"), work(c))
