"""Workloads of the 8-bit projection and of the 4-bit key/value cache.

Operators (the package's `w8a8_*` and `kv4_*` entry points):

  w8a8     y = (codes . w_codes^T) / a_scale[m] / w_scale[n], int8 x int8, either on codes that the program
           has ("gemm") or after RMSNorm and per-token absmax quantisation of x ("forward");
  append   the key and value rows of new tokens quantised to 4 bits into their pages, and read back;
  attend   softmax attention of query rows over the paged 4-bit cache.

The cache is uint8 [pages, kv heads, 64 * D + 1024]; a (page, head) block holds 64 tokens:
  [64][D / 2]  key codes, byte j of a token: dimension 2j in its low four bits, 2j + 1 in its high four,
  [64][D / 2]  value codes, the same,
  [64][2]      float32 (scale, minimum) of each key row, then the same of each value row;
a stored value is code * scale + minimum.  Position j of sequence b lies in page page_table[b, j // 64].
Sequence b owns the rows q_start[b] .. q_start[b + 1] - 1 of the new tokens, which are its last ones: row i of n is
position kv_lens[b] - n + i.

`run` computes them with elementary torch operations (own = False) or through the package (own = True).
"""
import math

import numpy as np
import torch

own = False

PAGE = 64
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
EPS = 1e-6


def listed():
    return [
        # one token through a 4096-wide projection of a decoder in bf16: latency and the weight stream
        dict(name="w8 token", op="w8", kind="forward", M=1, K=4096, N=4096, type="bf16"),
        # a few sequences decoding together through the sweep's 8192-wide projection
        dict(name="w8 13 tokens", op="w8", kind="gemm", M=13, K=8192, N=8192, type="f32"),
        # a prompt that is not a multiple of any tile, 16-bit in and out
        dict(name="w8 prompt", op="w8", kind="forward", M=2047, K=4096, N=8192, type="bf16"),
        # the sweep's largest token count
        dict(name="w8 16384 tokens", op="w8", kind="gemm", M=16384, K=4096, N=16384, type="f32"),
        # one decode step of 64 sequences: a row each, fp32 as the projections give them
        dict(name="append 64", op="append", B=64, n=1, L=4096, Hkv=8, D=128, type="f32"),
        # 64 prompts of 512 tokens at once
        dict(name="append 32768", op="append", B=64, n=512, L=512, Hkv=8, D=128, type="bf16"),
        # one sequence, short context: latency
        dict(name="attend one", op="attend", B=1, n=1, L=1021, Hq=16, Hkv=8, D=128, type="bf16", causal=True, window=0, ragged=False),
        # a serving batch of ragged lengths, fp32 in and out
        dict(name="attend 64 ragged", op="attend", B=64, n=1, L=8192, Hq=16, Hkv=8, D=128, type="f32", causal=True, window=0, ragged=True),
        # long contexts: the cache's stream
        dict(name="attend 16 long", op="attend", B=16, n=1, L=32768, Hq=16, Hkv=8, D=128, type="bf16", causal=True, window=0, ragged=False),
        # sliding-window layers of a model with one kv head of 256
        dict(name="attend 256 window", op="attend", B=256, n=1, L=4096, Hq=4, Hkv=1, D=256, type="f16", causal=True, window=512, ragged=True),
        # the last 4096 tokens of a prompt, given in pieces
        dict(name="attend chunk", op="attend", B=1, n=4096, L=12288, Hq=16, Hkv=8, D=128, type="bf16", causal=True, window=0, ragged=False),
        # a batch of texts to embed, both directions, every token of a text at once
        dict(name="attend texts", op="attend", B=64, n=512, L=512, Hq=4, Hkv=1, D=256, type="bf16", causal=False, window=0, ragged=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["w8", "w8", "append", "attend", "attend", "attend"])
    t = rng.choice(["f32", "bf16", "f16"])
    if kind == "w8":
        K = 128 * _log(rng, 2, 128)
        N = _log(rng, 64, 16384)
        M = _log(rng, 1, 16384)
        while M * K * N > 16384 * 4096 * 16384:
            M = max(1, M // 2)
        if rng.random() < 0.5:
            return dict(op="w8", kind="gemm", M=M, K=K, N=N, type=t)
        return dict(op="w8", kind="forward", M=M, K=K, N=N, type="bf16" if t == "f32" else t)  # 16 bits through a layer
    Hq, Hkv, D = rng.choice([(16, 8, 128), (4, 1, 256), (32, 8, 128), (8, 8, 128)])
    B = _log(rng, 1, 256)
    if kind == "append":
        n = _log(rng, 1, max(1, 32768 // B))
        return dict(op="append", B=B, n=n, L=n + _log(rng, 1, 2048), Hkv=Hkv, D=D, type=t)
    form = rng.choice(["one", "one", "few", "many"])
    if form == "many":
        B = _log(rng, 1, 64)
        n = _log(rng, 16, 4096)
        L = n + rng.choice([0, _log(rng, 1, 8192)])
        while B * n * Hq * L > 4096 * 16 * 12288 or B * n * Hq > 4096 * 16:
            B, n, L = max(1, B // 2), max(16, n * 3 // 4), max(16, L * 3 // 4)
        causal = rng.random() < 0.7
    else:
        n = 1 if form == "one" else rng.randint(2, 9)
        L = max(n, _log(rng, 1, 32768))
        while B * L * Hkv * D > 16 * 32768 * 8 * 128:
            B, L = max(1, B // 2), max(n, L * 3 // 4)
        causal = True
    window = rng.choice([0, 0, _log(rng, 16, 4096)]) if causal else 0
    return dict(op="attend", B=B, n=n, L=L, Hq=Hq, Hkv=Hkv, D=D, type=t, causal=causal, window=window, ragged=rng.random() < 0.5)


def _lengths(case):
    """(new tokens, tokens in the cache) of each sequence: a batch's lengths belong to the case, not to its data."""
    B, n, L = case["B"], case["n"], case["L"]
    r = np.random.RandomState(B * 131 + n * 17 + L)
    if not case.get("ragged"):
        return [n] * B, [L] * B
    lens = r.randint(1, L + 1, B)
    if n == L:  # whole texts
        return lens.tolist(), lens.tolist()
    return [n] * B, np.maximum(lens, n).tolist()


def _pairs(case):
    """Query-key pairs that the masks leave, and the cached tokens that any query of their sequence sees."""
    pairs = seen = 0
    for n, L in zip(*_lengths(case)):
        p = np.arange(L - n, L, dtype=np.int64)
        if not case["causal"]:
            pairs += n * L
            seen += L
            continue
        lo = np.maximum(0, p - case["window"] + 1) if case["window"] else np.zeros_like(p)
        pairs += int((p - lo + 1).sum())
        seen += int(L - lo[0])
    return pairs, seen


def work(case):
    size = 4 if case["type"] == "f32" else 2
    if case["op"] == "w8":
        M, K, N = case["M"], case["K"], case["N"]
        x = M * K * size + 4 * K if case["kind"] == "forward" else M * K + 4 * M
        return {"bytes": x + N * K + 4 * N + M * N * size, "flops": 2 * M * N * K}
    if case["op"] == "append":
        rows = case["B"] * case["n"] * case["Hkv"] * 2  # key and value rows
        D = case["D"]
        # read, pack; read the packed rows, give their values in fp32
        return {"bytes": rows * (D * size + 2 * (D // 2 + 8) + D * 4), "flops": rows * D * 6}
    pairs, seen = _pairs(case)
    rows = sum(_lengths(case)[0]) * case["Hq"] * case["D"]
    return {"bytes": 2 * rows * size + seen * case["Hkv"] * (case["D"] + 16), "flops": 4 * pairs * case["Hq"] * case["D"]}


def _quantise(x):
    """fp32 rows to (codes, scale, minimum): code = round(15 (x - min) / (max - min)), ties to even.  The quotient is
    taken in 64 bits, where a value next to the border of two codes falls on the right side of it."""
    lo, hi = x.amin(-1, keepdim=True), x.amax(-1, keepdim=True)
    span = hi - lo
    flat = span < 1e-30  # a constant row is its minimum
    scale = torch.where(flat, 0.0, span / 15.0)
    d = x.double() - lo.double()
    codes = torch.where(flat, 0.0, (d * 15.0) / (hi.double() - lo.double())).round().to(torch.uint8)
    return codes, scale.squeeze(-1), lo.squeeze(-1)


def _pack(codes):
    return codes[..., 0::2] | (codes[..., 1::2] << 4)


def _parts(cache, D):
    """Views of the cache's parts: codes [pages, heads, 64, D / 2], (scale, minimum) [pages, heads, 64, 2]."""
    c = PAGE * D // 2
    k, v = cache[..., :c], cache[..., c:2 * c]
    m = cache[..., 2 * c:].view(torch.float32)
    shape = cache.shape[:2]
    return (k.unflatten(-1, (PAGE, D // 2)), v.unflatten(-1, (PAGE, D // 2)),
            m[..., :2 * PAGE].reshape(*shape, PAGE, 2), m[..., 2 * PAGE:].reshape(*shape, PAGE, 2))


def _plan(case, g, dev):
    n, L = _lengths(case)
    B = len(n)
    per = [(x + PAGE - 1) // PAGE for x in L]
    most, pages = max(per), sum(per) + 3
    order = torch.randperm(pages, generator=g, device=dev).to(torch.int32)
    first = np.concatenate([[0], np.cumsum(per)[:-1]])
    at = torch.from_numpy(first[:, None] + np.arange(most)[None, :]).to(dev)
    used = torch.arange(most, device=dev)[None, :] < torch.tensor(per, device=dev)[:, None]
    table = torch.where(used, order[at.clamp(max=pages - 1)], torch.full_like(order[:1], -1))
    q_start = torch.tensor(np.concatenate([[0], np.cumsum(n)]), dtype=torch.int32, device=dev)
    lens = torch.tensor(L, dtype=torch.int32, device=dev)
    return dict(q_start=q_start, kv_lens=lens, table=table.contiguous(), pages=pages, T=sum(n), B=B, n=max(n), L=max(L))


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=dev)

    t = TYPES[case["type"]]
    s = dict(case=case)
    if case["op"] == "w8":
        M, K, N = case["M"], case["K"], case["N"]
        w = 0.02 * normal(N, K)
        w_scale = 127.0 / w.abs().amax(1)
        s.update(w=(w * w_scale[:, None]).round().clamp(-127, 127).to(torch.int8), w_scale=w_scale)
        x = normal(M, K)
        if case["kind"] == "forward":
            x[:, torch.randperm(K, generator=g, device=dev)[:max(1, K // 100)]] *= 20  # outlier features
            s.update(x=x.to(t), norm_w=1 + 0.1 * normal(K))
        else:
            a_scale = 127.0 / x.abs().amax(1)
            s.update(a=(x * a_scale[:, None]).round().clamp(-127, 127).to(torch.int8), a_scale=a_scale)
        return s
    D, Hkv = case["D"], case["Hkv"]
    plan = _plan(case, g, dev)
    s.update(plan)
    cache = torch.zeros(plan["pages"], Hkv, PAGE * D + 16 * PAGE, dtype=torch.uint8, device=dev)
    if case["op"] == "append":
        loud = 1 + 3 * (torch.rand(D, generator=g, device=dev) < 0.03)  # a few louder key channels
        s.update(cache=cache, k=(normal(plan["T"], Hkv, D) * loud).to(t), v=normal(plan["T"], Hkv, D).to(t))
        return s
    kc, vc, km, vm = _parts(cache, D)
    loud = 1 + 3 * (torch.rand(D, generator=g, device=dev) < 0.03)
    step = max(1, (1 << 27) // (Hkv * PAGE * D))  # pages at a time, to bound what the draws take
    for p in range(0, plan["pages"], step):
        e = min(plan["pages"], p + step)
        for codes, meta, gain in ((kc, km, loud), (vc, vm, 1.0)):
            c, sc, lo = _quantise(normal(e - p, Hkv, PAGE, D) * gain)
            codes[p:e] = _pack(c)
            meta[p:e, ..., 0], meta[p:e, ..., 1] = sc, lo
    s.update(cache=_joined(cache, kc, vc, km, vm, D), q=(normal(plan["T"], case["Hq"], D) * 1.5).to(t))
    return s


def _joined(cache, kc, vc, km, vm, D):
    c = PAGE * D // 2
    cache[..., :c], cache[..., c:2 * c] = kc.flatten(2), vc.flatten(2)
    cache[..., 2 * c:2 * c + 8 * PAGE] = km.flatten(2).contiguous().view(torch.uint8)
    cache[..., 2 * c + 8 * PAGE:] = vm.flatten(2).contiguous().view(torch.uint8)
    return cache


def _values(codes, meta):
    """Stored rows [..., D / 2] and their (scale, minimum) as fp32 values [..., D]."""
    c = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).float()
    return c * meta[..., :1] + meta[..., 1:]


def _run_w8(s):
    case = s["case"]
    t = TYPES[case["type"]]
    if own:
        import bitlinear_rmsnorm_token_gb300 as bn

        if case["kind"] == "forward":
            return bn.w8a8_forward(s["x"], s["norm_w"], s["w"], s["w_scale"], EPS)
        return bn.w8a8_gemm(s["a"], s["a_scale"], s["w"], s["w_scale"], y_dtype=t)
    if case["kind"] == "forward":
        x = s["x"].float()
        rstd = (1.0 / (x.double().square().mean(-1, keepdim=True) + EPS).sqrt()).float()
        xn = (x * rstd) * s["norm_w"]
        a_scale = 127.0 / xn.abs().amax(-1).clamp(min=1e-5)
        a = (xn * a_scale[:, None]).round().clamp(-128, 127)
    else:
        a, a_scale = s["a"].float(), s["a_scale"]
    acc = a @ s["w"].float().t()
    return ((acc * (1.0 / a_scale)[:, None]) * (1.0 / s["w_scale"])).to(t)


def _rows(s):
    """(sequence, position) of each new token."""
    t = torch.arange(s["T"], device=s["q_start"].device)
    b = torch.searchsorted(s["q_start"][1:].long(), t, right=True)
    at = s["kv_lens"][b] - (s["q_start"][b + 1] - s["q_start"][b]) + (t - s["q_start"][b])
    return b, at.long()


def _run_append(s):
    case = s["case"]
    D, Hkv = case["D"], case["Hkv"]
    if own:
        import bitlinear_rmsnorm_token_gb300 as bn

        bn.kv4_append(s["k"], s["v"], s["cache"], s["q_start"], s["kv_lens"], s["table"])
        return bn.kv4_read(s["cache"], s["T"], Hkv, D, s["q_start"], s["kv_lens"], s["table"])
    b, at = _rows(s)
    page = s["table"][b, at // PAGE].long()
    slot = at % PAGE
    c = PAGE * D // 2
    heads = torch.arange(Hkv, device=page.device)
    out = []
    for x, code_at, meta_at in ((s["k"], 0, 2 * c), (s["v"], c, 2 * c + 8 * PAGE)):
        codes, scale, lo = _quantise(x.float())
        meta = torch.stack([scale, lo], -1).view(torch.uint8)
        for part, start, width in ((_pack(codes), code_at, D // 2), (meta, meta_at, 8)):
            where = start + slot[:, None, None] * width + torch.arange(width, device=page.device)
            s["cache"][page[:, None, None], heads[None, :, None], where] = part
        got = []
        for start, width in ((code_at, D // 2), (meta_at, 8)):
            where = start + slot[:, None, None] * width + torch.arange(width, device=page.device)
            got.append(s["cache"][page[:, None, None], heads[None, :, None], where])
        out.append(_values(got[0], got[1].contiguous().view(torch.float32)))
    return tuple(out)


def _run_attend(s):
    case = s["case"]
    D, Hkv, Hq, n, L = case["D"], case["Hkv"], case["Hq"], s["n"], s["L"]
    if own:
        import bitlinear_rmsnorm_token_gb300 as bn

        return bn.kv4_attention(s["q"], s["cache"], Hkv, s["q_start"], s["kv_lens"], s["table"], n,
                                causal=case["causal"], window=case["window"])
    G, B, dev = Hq // Hkv, s["B"], s["q"].device
    blocks = s["cache"][s["table"].clamp(min=0).long()].transpose(1, 2)  # [B, heads, pages, bytes]
    kc, vc, km, vm = (x.flatten(2, 3) for x in _parts5(blocks, D))
    # queries, one padded row block per sequence
    count = (s["q_start"][1:] - s["q_start"][:-1]).long()
    i = torch.arange(n, device=dev)
    row = (s["q_start"][:-1].long()[:, None] + i).clamp(max=s["T"] - 1)
    q = s["q"].float()[row].unflatten(2, (Hkv, G)).permute(0, 2, 3, 1, 4).flatten(2, 3)  # [B, Hkv, G n, D]
    at = (s["kv_lens"].long() - count)[:, None] + i  # [B, n]
    j = torch.arange(kc.shape[2], device=dev)
    see = (j < s["kv_lens"].long()[:, None])[:, None, :].expand(B, n, -1)
    if case["causal"]:
        see = see & (j <= at[..., None])
        if case["window"]:
            see = see & (j > at[..., None] - case["window"])
    x = (q @ _values(kc, km).transpose(2, 3)) * (1.0 / math.sqrt(D))
    x = x.unflatten(2, (G, n)).masked_fill_(~see[:, None, None], float("-inf"))
    x = x - x.amax(-1, keepdim=True).clamp(min=-1e30)
    p = x.exp_()
    total = p.sum(-1, keepdim=True)
    o = p.flatten(2, 3) @ torch.where((j < s["kv_lens"].long()[:, None])[:, None, :, None], _values(vc, vm), 0.0)
    o = o.unflatten(2, (G, n)) / total.clamp(min=1e-30)
    b, _ = _rows(s)
    t = torch.arange(s["T"], device=dev)
    o = o.permute(0, 3, 1, 2, 4).flatten(2, 3)  # [B, n, Hq, D]
    return o[b, t - s["q_start"][b].long()].to(s["q"].dtype)


def _parts5(blocks, D):
    """_parts of gathered blocks [B, heads, pages, bytes]: [B, heads, pages, 64, ...]."""
    B, H, P, n = blocks.shape
    return (x.unflatten(0, (B, H)) for x in _parts(blocks.reshape(B * H, P, n), D))


def run(s):
    return {"w8": _run_w8, "append": _run_append, "attend": _run_attend}[s["case"]["op"]](s)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "w8":
        w = s["w"].double() / s["w_scale"].double()[:, None]
        if case["kind"] == "gemm":
            a = s["a"].double() / s["a_scale"].double()[:, None]
        else:
            x = s["x"].double()
            x = x * torch.rsqrt((x * x).sum(1, keepdim=True) / case["K"] + EPS) * s["norm_w"].double()
            top = x.abs().max(1, keepdim=True).values.clamp(min=1e-5)
            a = torch.round(x / top * 127) * top / 127
        return torch.cat([a[r:r + 4096] @ w.T for r in range(0, case["M"], 4096)])
    if case["op"] == "append":
        out = []
        for x in (s["k"].double(), s["v"].double()):
            lo = x.min(-1, keepdim=True).values
            width = x.max(-1, keepdim=True).values - lo
            out.append(torch.where(width > 0, torch.round(15 * (x - lo) / width) * width / 15 + lo, lo))
        return tuple(out)
    D, Hkv, Hq = case["D"], case["Hkv"], case["Hq"]
    G, half = Hq // Hkv, PAGE * D // 2
    out = torch.zeros(s["T"], Hq, D, dtype=torch.float64, device=s["q"].device)
    starts, lens = s["q_start"].tolist(), s["kv_lens"].tolist()
    for b, L in enumerate(lens):
        t0, t1 = starts[b], starts[b + 1]
        pages = s["table"][b, :(L + PAGE - 1) // PAGE].long()
        raw = s["cache"][pages]
        meta = raw[:, :, 2 * half:].contiguous().view(torch.float32).reshape(len(pages), Hkv, 2, PAGE, 2).double()
        kv = []
        for i in (0, 1):
            c = raw[:, :, i * half:(i + 1) * half].reshape(len(pages), Hkv, PAGE, D // 2)
            x = torch.empty(len(pages), Hkv, PAGE, D, dtype=torch.float64, device=c.device)
            x[..., 0::2], x[..., 1::2] = (c % 16).double(), (c // 16).double()
            x = x * meta[:, :, i, :, 0:1] + meta[:, :, i, :, 1:2]
            kv.append(x.transpose(0, 1).reshape(Hkv, -1, D)[:, :L])
        pos = torch.arange(L - (t1 - t0), L, device=raw.device)[:, None]
        key = torch.arange(L, device=raw.device)[None, :]
        ban = torch.zeros(t1 - t0, L, dtype=torch.bool, device=raw.device)
        if case["causal"]:
            ban = key > pos
            if case["window"]:
                ban = ban | (key <= pos - case["window"])
        for h in range(Hq):
            x = s["q"][t0:t1, h].double() @ kv[0][h // G].T / math.sqrt(D)
            out[t0:t1, h] = torch.softmax(x.masked_fill(ban, -math.inf), -1) @ kv[1][h // G]
    return out
