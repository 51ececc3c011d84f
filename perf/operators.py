"""Workloads of the 4-bit serving operators, with their plain forms.

Four operators, as the attention block of a decoder layer uses them in 4 bits:

  append      new tokens' keys and values quantized into an INT4 cache as they
              are written, and what was written read back;
  read        ragged ranges of an INT4 cache read back as 16- or 32-bit rows;
  attention   decode attention of a batch whose sequences share a long prefix:
              the prefix is cached once and multiplied once for all sequences,
              and every sequence attends its own cached tokens too;
  linear      activations quantized to MXFP4 (one plane, or two whose sum is
              close to 8 bits) and multiplied with MXFP4 weights.

With `own` false every operator is computed in elementary torch operations in
32 bits; with `own` true the library's entry points are called.
"""

import math
import random

import torch

own = False

D = 128                      # head dimension of the INT4 cache
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # one decode step of a batch: one new token a sequence
        dict(name="append_decode", op="append", seqs=32, hkv=8, cap=8192, new_lo=1, new_hi=1,
             start_hi=8000, dtype="bf16", fused=True),
        # a scheduler's step of chunked prefill: ragged pieces of several prompts
        dict(name="append_chunks", op="append", seqs=12, hkv=8, cap=8192, new_lo=1, new_hi=2047,
             start_hi=6000, dtype="bf16", fused=True),
        # rows handed back for a re-prefill of short prompts
        dict(name="read_short", op="read", seqs=16, hkv=8, cap=1024, new_lo=5, new_hi=401,
             start_hi=500, dtype="fp16"),
        # whole contexts read back for prefill attention over them
        dict(name="read_contexts", op="read", seqs=6, hkv=8, cap=32768, new_lo=9001, new_hi=32768,
             start_hi=0, dtype="bf16"),
        # a few chats on one system prompt: latency
        dict(name="attn_chat", op="attention", seqs=4, hq=32, hkv=8, prefix=1021, cap=128,
             len_lo=0, len_hi=61, dtype="bf16"),
        # a medium batch on a few-shot prompt
        dict(name="attn_fewshot", op="attention", seqs=32, hq=64, hkv=8, prefix=8189, cap=512,
             len_lo=1, len_hi=509, dtype="bf16"),
        # many samples of one long document, with long answers
        dict(name="attn_document", op="attention", seqs=64, hq=64, hkv=8, prefix=32768, cap=1024,
             len_lo=100, len_hi=1024, dtype="bf16"),
        # the largest: a long shared context and a large batch
        dict(name="attn_large", op="attention", seqs=128, hq=64, hkv=8, prefix=65537, cap=256,
             len_lo=0, len_hi=255, dtype="fp16"),
        # a decode step beyond the 16 tokens of the GEMV
        dict(name="linear_decode", op="linear", m=33, n=4096, k=4096, planes=2, dtype="bf16",
             strided=False),
        # a ragged prefill step, one plane, half of a fused projection's output as the input
        dict(name="linear_ragged", op="linear", m=509, n=4096, k=11008, planes=1, dtype="fp16",
             strided=True),
        # ordinary prefill, two planes
        dict(name="linear_prefill", op="linear", m=2048, n=25600, k=5120, planes=2, dtype="bf16",
             strided=False),
        # the largest prefill
        dict(name="linear_large", op="linear", m=8192, n=14336, k=4096, planes=2, dtype="bf16",
             strided=False),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "read", "attention", "attention", "linear", "linear"])
    dtype = rng.choice(["bf16", "bf16", "fp16"])
    if op == "append":
        seqs = _log_int(rng, 1, 48)
        cap = _log_int(rng, 64, 8192)
        most = max(1, min(cap // 2, 12000 // seqs))
        hi = _log_int(rng, 1, most)
        return dict(op=op, seqs=seqs, hkv=rng.choice([1, 2, 4, 8]), cap=cap,
                    new_lo=rng.choice([0, 1, hi]), new_hi=hi, start_hi=rng.randint(0, cap - hi),
                    dtype=rng.choice(["bf16", "fp16", "fp32"]), fused=rng.random() < 0.5)
    if op == "read":
        seqs = _log_int(rng, 1, 32)
        cap = _log_int(rng, 16, 32768)
        hi = _log_int(rng, 1, max(1, min(cap, 120000 // seqs)))
        return dict(op=op, seqs=seqs, hkv=rng.choice([1, 2, 4, 8]), cap=cap,
                    new_lo=rng.choice([0, 1, hi]), new_hi=hi, start_hi=rng.randint(0, cap - hi),
                    dtype=rng.choice(["bf16", "fp16", "fp32"]))
    if op == "attention":
        hkv = rng.choice([1, 2, 4, 8])
        hq = hkv * rng.choice([1, 2, 4, 8])
        seqs = _log_int(rng, 1, 128)
        prefix = _log_int(rng, 1, 65537)
        cap = _log_int(rng, 8, 1024)
        hi = rng.randint(0, cap)
        return dict(op=op, seqs=seqs, hq=hq, hkv=hkv, prefix=prefix, cap=cap,
                    len_lo=rng.randint(0, hi), len_hi=hi, dtype=dtype)
    n, k = 16 * _log_int(rng, 16, 1600), 128 * _log_int(rng, 4, 86)
    m = _log_int(rng, 1, min(8192, 8192 * 14336 * 4096 // (n * k)))
    return dict(op=op, m=m, n=n, k=k, planes=rng.choice([1, 2]), dtype=rng.choice(["bf16", "fp16", "fp32"]),
                strided=rng.random() < 0.5)


def _ragged(case):
    """The case's ragged lengths: counts (new tokens, or own tokens of an
    attention batch) and starts, the same for every seed."""
    r = random.Random(97 * case["seqs"] + case["cap"])
    if case["op"] == "attention":
        return [r.randint(case["len_lo"], case["len_hi"]) for _ in range(case["seqs"])], None
    counts = [r.randint(case["new_lo"], case["new_hi"]) for _ in range(case["seqs"])]
    return counts, [r.randint(0, case["start_hi"]) for _ in range(case["seqs"])]


def work(case):
    if case["op"] == "linear":
        m, n, k = case["m"], case["n"], case["k"]
        size = 4 if case["dtype"] == "fp32" else 2
        return {"bytes": m * k * size + n * k // 2 + n * k // 32 + m * n * 2,
                "flops": 2 * m * n * k}
    counts, _ = _ragged(case)
    row = D // 2 + 4                                     # codes, scale and zero of one row
    if case["op"] == "attention":
        keys = case["prefix"] + sum(counts)
        products = case["seqs"] * case["prefix"] + sum(counts)
        return {"bytes": 2 * case["hkv"] * keys * row + 2 * case["seqs"] * case["hq"] * D * 2,
                "flops": 4 * products * case["hq"] * D}
    size = 4 if case["dtype"] == "fp32" else 2
    rows = 2 * sum(counts) * case["hkv"]
    # append: rows read, cache written, and the cache read back as rows
    times = 2 if case["op"] == "append" else 1
    return {"bytes": times * rows * (D * size + row), "flops": times * rows * D * 3}


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------

def _int4_plain(x):
    """One INT4 group a row of x fp32 [..., D]: codes int32, scales and zeros fp16."""
    lo = x.amin(-1, keepdim=True).clamp(max=0.0)
    hi = x.amax(-1, keepdim=True).clamp(min=0.0)
    fifteen = torch.full_like(lo, 15.0)                  # a tensor: an IEEE division
    s = ((hi - lo) / fifteen).half()
    empty = s == 0
    lo = torch.where(empty, torch.full_like(lo, -1.0), lo)
    s = torch.where(empty, (torch.full_like(lo, 2.0) / fifteen).half(), s)
    sf = s.float()
    z = torch.round(-lo / sf).clamp(0, 15)
    q = (torch.round(x / sf) + z).clamp(0, 15)
    return q.to(torch.int32), s.squeeze(-1), z.squeeze(-1).half()


def _or_nibbles(c):
    """int32 [..., 8] codes -> int32 [...], element i in nibble i."""
    w = c[..., 0].clone()
    for i in range(1, 8):
        w |= c[..., i] << (4 * i)
    return w


def _nibbles(w):
    """int32 [...] -> int32 [..., 8]."""
    return torch.stack([(w >> (4 * i)) & 15 for i in range(8)], dim=-1)


def _pack_cache(k, v):
    """Caches of fp32 rows [B, H, L, D]: keys a token a row, values in blocks of 8 tokens."""
    b, h, n, d = k.shape
    kc, ks, kz = _int4_plain(k)
    kq = _or_nibbles(kc.view(b, h, n, d // 8, 8))
    del kc
    vc, vs, vz = _int4_plain(v)
    pad = -n % 8
    if pad:
        vc = torch.cat([vc, vc.new_zeros(b, h, pad, d)], dim=2)
    vq = _or_nibbles(vc.view(b, h, (n + pad) // 8, 8, d).transpose(3, 4))
    return (kq, ks, kz), (vq, vs, vz)


def _codes_plain(cache, is_value, n):
    """Codes fp32 [B, H, n, D] of a cache's first n tokens."""
    w = cache[0]
    b, h = w.shape[:2]
    if not is_value:
        return _nibbles(w[:, :, :n]).reshape(b, h, n, D).float()
    nb = (n + 7) // 8
    return _nibbles(w[:, :, :nb]).transpose(3, 4).reshape(b, h, nb * 8, D)[:, :, :n].float()


def _dequant_plain(cache, is_value, n):
    _, s, z = cache
    return (_codes_plain(cache, is_value, n) - z[:, :, :n, None].float()) * \
        s[:, :, :n, None].float()


def _positions(offsets, starts, total):
    """Sequence and cache position of each of the packed tokens."""
    seqs = starts.numel()
    token = torch.arange(total, device=starts.device)
    seq = torch.repeat_interleave(torch.arange(seqs, device=starts.device),
                                  offsets[1:] - offsets[:-1], output_size=total)
    return seq, token - offsets[seq].long() + starts[seq].long()


def _append_plain(k, v, k_cache, v_cache, starts, offsets):
    total, h, d = k.shape
    seq, pos = _positions(offsets, starts, total)
    seq, pos = seq[:, None], pos[:, None]
    head = torch.arange(h, device=k.device)[None]
    kc, ks, kz = _int4_plain(k.float())
    k_cache[0][seq, head, pos] = _or_nibbles(kc.view(total, h, d // 8, 8))
    k_cache[1][seq, head, pos] = ks
    k_cache[2][seq, head, pos] = kz
    vc, vs, vz = _int4_plain(v.float())
    v_cache[1][seq, head, pos] = vs
    v_cache[2][seq, head, pos] = vz
    # up to 8 tokens share a word: add every token's change of its own nibble
    blk, shift = pos // 8, (4 * (pos % 8))[..., None].to(torch.int32)
    old = (v_cache[0][seq, head, blk] >> shift) & 15
    v_cache[0].index_put_((seq, head, blk), (vc - old) << shift, accumulate=True)


def _read_plain(k_cache, v_cache, starts, offsets, total, dtype):
    seq, pos = _positions(offsets, starts, total)
    seq, pos = seq[:, None], pos[:, None]
    out = []
    for cache, is_value in ((k_cache, False), (v_cache, True)):
        w, s, z = cache
        head = torch.arange(w.shape[1], device=w.device)[None]
        if is_value:
            c = (w[seq, head, pos // 8] >> (4 * (pos % 8))[..., None].to(torch.int32)) & 15
        else:
            c = _nibbles(w[seq, head, pos]).reshape(total, w.shape[1], D)
        x = (c.float() - z[seq, head, pos][..., None].float()) * s[seq, head, pos][..., None].float()
        out.append(x.to(dtype))
    return out


def _attention_plain(q, prefix_k, prefix_v, k_cache, v_cache, lengths, prefix_len):
    b, hq, d = q.shape
    hkv = k_cache[1].shape[1]
    r = hq // hkv
    cap = k_cache[1].shape[2]
    qf = q.float().view(b, hkv, r, d) * (1.0 / math.sqrt(d))
    kp = _dequant_plain(prefix_k, False, prefix_len)[0]            # [Hkv, P, D]
    rows = qf.transpose(0, 1).reshape(hkv, b * r, d)
    sp = torch.matmul(rows, kp.transpose(1, 2))                    # [Hkv, B R, P]
    del kp
    ss = torch.matmul(qf, _dequant_plain(k_cache, False, cap).transpose(2, 3))
    dead = torch.arange(cap, device=q.device)[None] >= lengths[:, None]
    ss.masked_fill_(dead[:, None, None], -math.inf)
    ss = ss.transpose(0, 1).reshape(hkv, b * r, cap)
    m = torch.maximum(sp.amax(-1, keepdim=True), ss.amax(-1, keepdim=True))
    sp.sub_(m).exp_()
    ss.sub_(m).exp_()
    total = sp.sum(-1, keepdim=True) + ss.sum(-1, keepdim=True)
    out = torch.matmul(sp, _dequant_plain(prefix_v, True, prefix_len)[0])
    del sp
    own_part = torch.matmul(ss.view(hkv, b, r, cap).transpose(0, 1),
                            _dequant_plain(v_cache, True, cap))
    out = (out + own_part.transpose(0, 1).reshape(hkv, b * r, d)) / total
    return out.view(hkv, b, r, d).transpose(0, 1).reshape(b, hq, d).to(q.dtype)


def _mxfp4_plain(x):
    """MXFP4 values of x fp32 [M, K] (the element values, and exponents [M, K / 32])."""
    blocks = x.view(x.shape[0], -1, 32)
    mant, exp = torch.frexp(blocks.abs().amax(-1))
    # the smallest e with amax <= 6 * 2^e: 6 = 0.75 * 2^3
    e = torch.where(mant <= 0.75, exp - 3, exp - 2)
    e = torch.where(mant == 0, torch.zeros_like(e), e).clamp(-127, 127)
    v = torch.ldexp(blocks, -e[..., None])
    a = v.abs()
    a = torch.where(a < 2, torch.round(a * 2) * 0.5,
                    torch.where(a < 4, torch.round(a), torch.round(a * 0.5) * 2))
    return a.copysign(v), e


def _mxfp4_value(v, e):
    return torch.ldexp(v, e[..., None]).reshape(v.shape[0], -1)


def _mxfp4_pack(v, e):
    """Codes uint8 [M, K / 2] (element 2j in the low nibble) and scale bytes."""
    a = v.abs()
    code = torch.where(a < 2, a * 2, torch.where(a < 4, a + 2, a * 0.5 + 4)).to(torch.uint8)
    code |= ((v < 0) & (code != 0)).to(torch.uint8) << 3
    code = code.view(v.shape[0], -1)
    return code[:, 0::2] | (code[:, 1::2] << 4), (e + 127).to(torch.uint8)


def _mxfp4_unpack(codes, scales):
    lut = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=codes.device)
    c = torch.stack([codes & 15, codes >> 4], dim=-1).view(codes.shape[0], -1, 32).int()
    v = torch.where(c >= 8, -lut[c & 7], lut[c & 7])
    return _mxfp4_value(v, scales.int() - 127)


def _linear_plain(x, codes, scales, planes):
    xf = x.float()
    hat = _mxfp4_value(*_mxfp4_plain(xf))
    if planes == 2:
        hat = hat + _mxfp4_value(*_mxfp4_plain(xf - hat))
    return torch.matmul(hat, _mxfp4_unpack(codes, scales).t()).to(torch.bfloat16)


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(1234567 + 7919 * int(seed))
    return g


def _kv_rows(g, b, h, n):
    """Keys N(0, 0.5) with a few channels of a head scaled up, values N(0, 1): fp32 [B, H, n, D]."""
    k = torch.randn(b, h, n, D, generator=g, device="cuda") * 0.5
    gain = torch.ones(h, D, device="cuda")
    gain.scatter_(1, torch.randint(0, D, (h, 5), generator=g, device="cuda"), 8.0)
    k *= gain[None, :, None]
    return k, torch.randn(b, h, n, D, generator=g, device="cuda")


def prepare(case, seed):
    g = _generator(seed)
    st = dict(case=dict(case))
    if case["op"] == "linear":
        m, n, k = case["m"], case["n"], case["k"]
        wide = torch.randn(m, 2 * k if case["strided"] else k, generator=g, device="cuda")
        wide[:, torch.randint(0, k, (max(1, k // 100),), generator=g, device="cuda")] *= 20.0
        st["x"] = wide.to(DTYPES[case["dtype"]])[:, :k]
        w = torch.randn(n, k, generator=g, device="cuda") * 0.02
        st["codes"], st["scales"] = _mxfp4_pack(*_mxfp4_plain(w))
        if own:
            from bit_weight_quantized_weights_b200 import binding as wq
            st["workspace"] = wq.mx_gemm_workspace(m, n, k, case["planes"], "cuda")
        return st
    b, h, cap = case["seqs"], case["hkv"], case["cap"]
    counts, starts = _ragged(case)
    k, v = _kv_rows(g, b, h, cap)
    st["k_cache"], st["v_cache"] = _pack_cache(k, v)
    del k, v
    if case["op"] == "attention":
        hq, p = case["hq"], case["prefix"]
        st["prefix_k"], st["prefix_v"] = _pack_cache(*_kv_rows(g, 1, h, p))
        st["q"] = torch.randn(b, hq, D, generator=g, device="cuda").to(DTYPES[case["dtype"]])
        st["lengths"] = torch.tensor(counts, dtype=torch.int32, device="cuda")
        if own:
            from bit_weight_quantized_weights_b200 import binding as wq
            st["workspace"] = wq.prefix_attention_workspace(b, hq, h, p, cap, D, "cuda")
        return st
    st["total"] = total = sum(counts)
    st["starts"] = torch.tensor(starts, dtype=torch.int32, device="cuda")
    edges = [0]
    for c in counts:
        edges.append(edges[-1] + c)
    st["offsets"] = torch.tensor(edges, dtype=torch.int32, device="cuda")
    if case["op"] == "append":
        dt = DTYPES[case["dtype"]]
        k, v = _kv_rows(g, 1, h, total)
        k, v = k[0].transpose(0, 1).to(dt), v[0].transpose(0, 1).to(dt)     # [T, H, D]
        if case["fused"]:
            # keys and values are slices of one projection's output
            both = torch.cat([k, v], dim=1).contiguous()
            st["k"], st["v"] = both[:, :h], both[:, h:]
        else:
            st["k"], st["v"] = k.contiguous(), v.contiguous()
    return st


def run(state):
    case = state["case"]
    op = case["op"]
    if own:
        from bit_weight_quantized_weights_b200 import binding as wq
        if op == "linear":
            planes, scales = wq.wq_mx_quantize_planes(state["x"], case["planes"])
            return wq.wq_mx_gemm(planes, scales, case["n"], state["codes"], state["scales"],
                                 workspace=state["workspace"])
        if op == "attention":
            return wq.wq_prefix_attention(state["q"], state["prefix_k"], state["prefix_v"],
                                          state["k_cache"], state["v_cache"], state["lengths"],
                                          workspace=state["workspace"])
        if op == "append":
            wq.wq_kv_append(state["k"], state["v"], state["k_cache"], state["v_cache"],
                            state["starts"], state["offsets"])
        out = wq.wq_kv_read(state["k_cache"], state["v_cache"], state["starts"],
                            state["offsets"], state["total"], dtype=DTYPES[case["dtype"]])
    else:
        if op == "linear":
            return _linear_plain(state["x"], state["codes"], state["scales"], case["planes"])
        if op == "attention":
            return _attention_plain(state["q"], state["prefix_k"], state["prefix_v"],
                                    state["k_cache"], state["v_cache"], state["lengths"],
                                    case["prefix"])
        if op == "append":
            _append_plain(state["k"], state["v"], state["k_cache"], state["v_cache"],
                          state["starts"], state["offsets"])
        out = _read_plain(state["k_cache"], state["v_cache"], state["starts"], state["offsets"],
                          state["total"], DTYPES[case["dtype"]])
    if op == "append":
        # the scales and zeros of the whole caches: the rows around stay as they were
        return list(out) + list(state["k_cache"][1:]) + list(state["v_cache"][1:])
    return list(out)


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def _exact_rows(words, scales, zeros, is_value, first, n):
    """fp64 rows first .. first + n - 1 of one (sequence, head) of a cache."""
    at = torch.arange(first, first + n, device=words.device)
    d = torch.arange(D, device=words.device)
    if is_value:
        c = (words[at // 8] >> (4 * (at % 8)).to(torch.int32)[:, None]) & 15
    else:
        c = (words[at][:, d // 8] >> (4 * (d % 8)).to(torch.int32)[None]) & 15
    return (c.double() - zeros[at].double()[:, None]) * scales[at].double()[:, None]


def _exact_group(x):
    """Scale, zero and the values of the codes of rows x (any 16- or 32-bit
    type): the roundings of the definition, each made from a 64-bit value."""
    def rn32(t):
        return t.to(torch.float32).double()
    x = x.double()
    lo = torch.minimum(x.min(-1)[0], torch.zeros((), dtype=x.dtype, device=x.device))
    hi = torch.maximum(x.max(-1)[0], torch.zeros((), dtype=x.dtype, device=x.device))
    s = rn32(rn32(hi - lo) / 15).half()
    none = s == 0
    lo = torch.where(none, -torch.ones_like(lo), lo)
    s = torch.where(none, torch.full_like(s, 2 / 15), s)
    sd = s.double()
    z = rn32(-lo / sd).round().clamp(0, 15)
    q = (rn32(x / sd[..., None]).round() + z[..., None]).clamp(0, 15)
    return s, z.half(), (q - z[..., None]) * sd[..., None]


def _exact_mx(x):
    """MXFP4 of x fp64: x's blocks of 32 rounded to the element values, in 64 bits."""
    blocks = x.view(x.shape[0], -1, 32)
    top = blocks.abs().amax(-1, keepdim=True)
    unit = torch.exp2(torch.ceil(torch.log2(top / 6)))
    unit = torch.where(6 * unit < top, unit * 2, unit)
    unit = torch.where(6 * (unit / 2) >= top, unit / 2, unit)
    unit = torch.where(top > 0, unit, torch.ones_like(unit)).clamp(2.0 ** -127, 2.0 ** 127)
    a = blocks.abs() / unit
    out = torch.zeros_like(a)
    grid = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
    for i in range(1, 8):
        mid = (grid[i - 1] + grid[i]) / 2
        up = a >= mid if i % 2 == 0 else a > mid         # a tie goes to the even code
        out = torch.where(up, torch.full_like(out, grid[i]), out)
    return (out * unit * torch.sign(blocks)).view(x.shape)


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "linear":
        x = st["x"].double().contiguous()
        hat = _exact_mx(x)
        if case["planes"] == 2:
            hat = hat + _exact_mx(x - hat)
        c, value = st["codes"].long(), [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
        table = torch.tensor(value + [-t for t in value], dtype=torch.float64, device="cuda")
        w = torch.stack([table[c % 16], table[c // 16]], dim=2).view(case["n"], -1, 32)
        w = w * torch.exp2(st["scales"].double() - 127)[..., None]
        return hat @ w.view(case["n"], case["k"]).t()
    counts, starts = _ragged(case)
    if op == "attention":
        b, hkv, r = case["seqs"], case["hkv"], case["hq"] // case["hkv"]
        q = st["q"].double().view(b, hkv, r, D)
        out = torch.empty(b, hkv, r, D, dtype=torch.float64, device="cuda")
        for h in range(hkv):
            kp = _exact_rows(*[t[0, h] for t in st["prefix_k"]], False, 0, case["prefix"])
            vp = _exact_rows(*[t[0, h] for t in st["prefix_v"]], True, 0, case["prefix"])
            for i in range(b):
                ks = _exact_rows(*[t[i, h] for t in st["k_cache"]], False, 0, counts[i])
                vs = _exact_rows(*[t[i, h] for t in st["v_cache"]], True, 0, counts[i])
                p = torch.softmax(torch.cat([q[i, h] @ kp.t(), q[i, h] @ ks.t()], 1) /
                                  math.sqrt(D), dim=1)
                out[i, h] = p[:, :case["prefix"]] @ vp + p[:, case["prefix"]:] @ vs
        return out.view(b, case["hq"], D)
    rows = [[], []]
    if op == "read":
        for j, (cache, is_value) in enumerate(((st["k_cache"], False), (st["v_cache"], True))):
            for i, (n, first) in enumerate(zip(counts, starts)):
                rows[j].append(torch.stack(
                    [_exact_rows(*[t[i, h] for t in cache], is_value, first, n)
                     for h in range(case["hkv"])], dim=1))
        return [torch.cat(t) for t in rows]
    out, held = [], []
    for new, cache in ((st["k"], st["k_cache"]), (st["v"], st["v_cache"])):
        s, z, x = _exact_group(new)
        at = 0
        for i, (n, first) in enumerate(zip(counts, starts)):
            cache[1][i, :, first:first + n] = s[at:at + n].t()
            cache[2][i, :, first:first + n] = z[at:at + n].t()
            at += n
        out.append(x)
        held += [cache[1], cache[2]]
    return out + held
