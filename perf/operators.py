"""The operators around a rotated and a 4-bit paged KV cache, as cases that can be timed.

Three operators:

* ``append``: a step's queries, keys and values enter the attention: an optional
  RMS norm of every query and key head, the position rotation, the rotated
  queries written out, and keys and values stored at their slots of the paged
  pools (16-bit elements, E4M3 codes or 4-bit codes).
* ``write4``: 16-bit keys and values stored as 4-bit codes at their slots, and
  the same rows read back as 16-bit values.
* ``decode4``: single-query attention over 4-bit pools.

A 4-bit pool holds E2M1 codes (0, .5, 1, 1.5, 2, 3, 4, 6 and their negatives)
with one E4M3 scale for every 16 consecutive head_dim values of a token and one
float32 scale for the tensor: value = code * scale16 * scale.  Pools are uint8
[num_blocks][num_kv_heads][B * 9 D / 16]; the bytes of a (block, head) are the
codes [B][D / 2] (the even element in the low nibble), then the scales
[B / 4][D / 16][4], the last index being the token's position modulo 4.

With ``own`` false the operators run in their plain form, elementary torch
operations in 32 bits; with ``own`` true they are this package's calls.
"""
import math

import numpy as np
import torch

own = False

DT = {"fp16": torch.float16, "bf16": torch.bfloat16}
EPS = 1e-6


# ---------------------------------------------------------------------------
# The cases
# ---------------------------------------------------------------------------

def _append(name, Hq, Hkv, D, B, dtype, seqs, new, past, pool, **more):
    c = dict(name=name, op="append", Hq=Hq, Hkv=Hkv, D=D, B=B, dtype=dtype, seqs=seqs, new=new,
             past=past, pool=pool, rot=D, interleaved=False, norm=False, len_seed=1)
    c.update(more)
    return c


def _write4(name, Hkv, D, B, dtype, seqs, new, past, **more):
    c = dict(name=name, op="write4", Hq=0, Hkv=Hkv, D=D, B=B, dtype=dtype, seqs=seqs, new=new,
             past=past, pool="e2m1", rot=0, interleaved=False, norm=False, len_seed=2)
    c.update(more)
    return c


def _decode4(name, Hq, Hkv, D, B, dtype, seqs, lens, **more):
    c = dict(name=name, op="decode4", Hq=Hq, Hkv=Hkv, D=D, B=B, dtype=dtype, seqs=seqs, lens=lens,
             lo=0, hi=0, window=0, sigma=1.0, len_seed=3)
    c.update(more)
    return c


def listed():
    return [
        # the smallest step: the tiny workload's four sequences, one new token each
        _append("append tiny", 8, 8, 64, 4, "fp16", 4, 1, 40, "16"),
        # one decode step of the Llama-3-8B layer's batch, heads normed
        _append("append llama3-8b step", 32, 8, 128, 16, "bf16", 256, 1, 800, "16", norm=True),
        # the chunked-prefill step: 16 prompts of 512 new tokens
        _append("append llama3-8b prefill", 32, 8, 128, 16, "bf16", 16, 512, 6144, "16",
                norm=True),
        # ragged prompts without grouped heads into an E4M3 cache, half of each head rotated,
        # neighbours paired
        _append("append llama2-7b e4m3", 32, 32, 128, 16, "fp16", 7, 277, 1500, "e4m3", rot=64,
                interleaved=True),
        # the 70B-class layer's step into a 4-bit cache, and a prompt step's
        _append("append 70b 4-bit step", 64, 8, 128, 16, "bf16", 32, 1, 32767, "e2m1"),
        _append("append llama3-8b 4-bit", 32, 8, 128, 16, "bf16", 16, 512, 6144, "e2m1"),
        # a shared prefix moved to 4 bits (Qwen2-0.5B's heads), and a prompt step's rows
        _write4("write4 qwen2 prefix", 2, 64, 16, "fp16", 1, 1800, 0),
        _write4("write4 llama3-8b", 8, 128, 16, "bf16", 16, 512, 6144),
        # decode: the tiny lengths, the Llama-3-8B batch, no grouped heads, the 70B-class layer
        _decode4("decode4 tiny", 8, 8, 64, 4, "fp16", 4, "tiny"),
        _decode4("decode4 llama3-8b", 32, 8, 128, 16, "bf16", 256, "lognormal", sigma=0.5),
        _decode4("decode4 llama2-7b", 32, 32, 128, 16, "fp16", 64, "uniform", lo=1, hi=2048),
        _decode4("decode4 70b long", 64, 8, 128, 16, "bf16", 32, "uniform", lo=16384, hi=32768),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    dtype = rng.choice(("bf16", "fp16"))
    D = rng.choice((64, 128, 128))
    kind = rng.choice(("append", "append", "write4", "decode4", "decode4", "decode4"))
    len_seed = rng.randrange(1 << 20)
    Hkv = rng.choice((1, 2, 3, 4, 5, 8, 8, 16, 32))
    if kind == "decode4":
        G = rng.choice((1, 2, 3, 4, 5, 7, 8, 8, 12, 16))
        while Hkv * G > 64:
            Hkv = max(1, Hkv // 2)
        B = rng.choice((4, 8, 16, 16, 32, 64, 256))
        seqs = _log_int(rng, 1, 256)
        # padded lengths within the largest listed case's
        most = min(32768, (32 * 32768 * 8 * 128) // (seqs * Hkv * D))
        hi = _log_int(rng, 1, most)
        lo = rng.choice((0, 1, hi // 2))
        window = rng.choice((0, 0, 0, _log_int(rng, 1, 4096)))
        return dict(op="decode4", Hq=Hkv * G, Hkv=Hkv, D=D, B=B, dtype=dtype, seqs=seqs,
                    lens="uniform", lo=min(lo, hi), hi=hi, window=window,
                    sigma=rng.choice((0.5, 1.0)), len_seed=len_seed)
    seqs = _log_int(rng, 1, 64)
    new = _log_int(rng, 1, max(1, 8192 // seqs))
    past = _log_int(rng, 1, 8192)
    if kind == "write4":
        while Hkv * D > 1024:
            Hkv //= 2
        return dict(op="write4", Hq=0, Hkv=Hkv, D=D, B=rng.choice((4, 8, 16, 32, 128)),
                    dtype=dtype, seqs=seqs, new=new, past=past, pool="e2m1", rot=0,
                    interleaved=False, norm=False, len_seed=len_seed)
    G = rng.choice((1, 2, 4, 7, 8))
    while Hkv > 1 and Hkv * (G + 2) * D > 48 * 128:
        Hkv //= 2
    pool = rng.choice(("16", "16", "e4m3", "e2m1"))
    past = min(past, max(1, (1 << 27) // (seqs * Hkv * D)))
    return dict(op="append", Hq=Hkv * G, Hkv=Hkv, D=D, B=rng.choice((4, 8, 16, 32, 128)),
                dtype=dtype, seqs=seqs, new=new, past=past, pool=pool,
                rot=rng.choice((D, D, D // 2, 16)), interleaved=rng.random() < 0.3,
                norm=pool == "16" and rng.random() < 0.5, len_seed=len_seed)


def _lengths(case):
    """The sequences' lengths of a decode case: plain integers, the same for every seed."""
    rng = np.random.default_rng(case["len_seed"])
    n = case["seqs"]
    if case["lens"] == "tiny":
        return np.array([7, 8, 9, 33], np.int32)
    if case["lens"] == "lognormal":
        s = 0.632
        t = np.rint(rng.lognormal(math.log(400.0) - s * s / 2, s, size=n))
        return np.clip(t, 16, 4096).astype(np.int32)
    return rng.integers(case["lo"], case["hi"], size=n, endpoint=True).astype(np.int32)


def _tokens(case):
    """(sequence, position) of every new token and the sequences' lengths after them."""
    rng = np.random.default_rng(case["len_seed"])
    n = case["seqs"]
    new = np.full(n, case["new"], np.int64)
    if case["new"] > 1 and n > 1 and case["len_seed"] != 1:
        new = rng.integers(1, case["new"], size=n, endpoint=True)   # ragged
    past = rng.integers(0, case["past"], size=n, endpoint=True)
    seq = np.repeat(np.arange(n, dtype=np.int32), new)
    pos = np.concatenate([np.arange(p, p + c) for p, c in zip(past, new)]).astype(np.int32)
    return seq, pos, (past + new).astype(np.int64)


def _row_bytes(case):
    """Bytes of one token's K or V row of one head in the pool."""
    D = case["D"]
    return {"16": 2 * D, "e4m3": D, "e2m1": 9 * D // 16}[case.get("pool", "e2m1")]


def work(case):
    D, Hq, H = case["D"], case["Hq"], case["Hkv"]
    if case["op"] == "decode4":
        T = _lengths(case).astype(np.int64)
        if case["window"]:
            T = np.minimum(T, case["window"])
        blocks = int(np.sum(-(-T // case["B"])))
        t = int(T.sum())
        return {"bytes": t * H * 2 * _row_bytes(case) + 4 * case["seqs"] * Hq * D + 4 * blocks
                + 4 * case["seqs"], "flops": 4 * t * Hq * D}
    seq, pos, _ = _tokens(case)
    n = len(seq)
    bytes_ = n * (2 * Hq + 2 * H) * D * 2 + n * 2 * H * _row_bytes(case)    # q, k, v; q, K, V out
    bytes_ += n * 12 + len(np.unique(pos)) * case["rot"] * 4    # sequence, position, table; angles
    flops = n * (Hq + H) * case["rot"] * 3 + (n * (Hq + H) * D * 4 if case["norm"] else 0)
    if case["pool"] == "e2m1":
        bytes_ += n * 2 * H * (_row_bytes(case) + 2 * D)        # read back as 16-bit rows
        flops += n * 2 * H * D * 3
    return {"bytes": bytes_, "flops": flops}


# ---------------------------------------------------------------------------
# 4-bit pools, plain form
# ---------------------------------------------------------------------------

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _e4m3(x):
    """x >= 0 in 32 bits, rounded to the nearest E4M3 value (at most 448)."""
    return x.clamp(max=448.0).to(torch.float8_e4m3fn)


def _quantize4(x, s):
    """x [..., D] in 32 bits, s the tensor's scale (a 0-d tensor in 32 bits) -> codes uint8
    [..., D / 2], scales uint8 [..., D / 16]."""
    g = x.reshape(x.shape[:-1] + (x.shape[-1] // 16, 16))
    s8 = _e4m3(g.abs().amax(-1) / (s * 6.0))
    d = (s8.float() * s)[..., None]
    a = torch.where(d > 0, g.abs() / d, torch.zeros_like(g))
    code = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5)
            + (a >= 3.5) + (a > 5.0))
    code = code | ((g < 0).to(torch.uint8) << 3)
    code = code.reshape(x.shape)
    return code[..., 0::2] | (code[..., 1::2] << 4), s8.view(torch.uint8)


def _views4(pool, D, B):
    """The codes [nb, H, B, D / 2] and scales [nb, H, B / 4, D / 16, 4] of a 4-bit pool."""
    nb, H = pool.shape[:2]
    P = B * 9 * D // 16
    flat = pool.view(-1)
    codes = flat.as_strided((nb, H, B, D // 2), (H * P, P, D // 2, 1))
    scales = flat.as_strided((nb, H, B // 4, D // 16, 4), (H * P, P, D // 4, 4, 1), B * D // 2)
    return codes, scales


def _byte_values(dev):
    """[256, 2]: the two E2M1 values of every byte."""
    one = torch.tensor(E2M1 + tuple(-v for v in E2M1), dtype=torch.float32, device=dev)
    byte = torch.arange(256, device=dev)
    return torch.stack((one[byte & 15], one[byte >> 4]), -1)


def _values4(codes, scales, two):
    """codes [..., D / 2], scales [..., D / 16] -> code * scale16 [..., D] in 32 bits."""
    v = two[codes.int()]                                        # [..., D / 2, 2]
    s = scales.view(torch.float8_e4m3fn).float()
    v = v.reshape(s.shape + (16,)) * s[..., None]
    return v.reshape(codes.shape[:-1] + (codes.shape[-1] * 2,))


def _store4(pool, x, blk, row, scale, D, B):
    codes, scales = _views4(pool, D, B)
    c, s = _quantize4(x, scale)
    codes[blk, :, row] = c
    scales[blk, :, row // 4, :, row % 4] = s


def _load4(pool, blk, row, scale, D, B, dtype, two):
    codes, scales = _views4(pool, D, B)
    v = _values4(codes[blk, :, row], scales[blk, :, row // 4, :, row % 4], two)
    return (v * scale).to(dtype)


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

def _device():
    return "cuda" if torch.cuda.is_available() else "cpu"


def _tables(lens, B, num_blocks, g, dev):
    """Blocks of a random permutation of the pool, sequence by sequence; -1 past the end."""
    need = -(-np.asarray(lens, np.int64) // B)
    stride = max(1, int(need.max()))
    perm = torch.randperm(num_blocks, generator=g, device=dev).int()
    start = torch.from_numpy(np.concatenate([[0], np.cumsum(need)[:-1]])).to(dev)
    col = torch.arange(stride, device=dev)
    idx = (start[:, None] + col[None]).clamp(max=num_blocks - 1)
    inside = col[None] < torch.from_numpy(need).to(dev)[:, None]
    return torch.where(inside, perm[idx], torch.full_like(perm[idx], -1)).contiguous()


def _pool4(num_blocks, H, B, D, sigma, scale, g, dev):
    """A 4-bit pool of quantized N(0, sigma^2) values."""
    pool = torch.empty(num_blocks, H, B * 9 * D // 16, dtype=torch.uint8, device=dev)
    codes, scales = _views4(pool, D, B)
    step = max(1, (1 << 26) // (H * B * D))
    scale = torch.tensor(scale, dtype=torch.float32, device=dev)
    for b in range(0, num_blocks, step):
        n = min(step, num_blocks - b)
        c, s = _quantize4(torch.randn(n, H, B, D, generator=g, device=dev) * sigma, scale)
        codes[b:b + n] = c
        scales[b:b + n] = s.reshape(n, H, B // 4, 4, D // 16).transpose(-1, -2)
    return pool


def prepare(case, seed):
    dev = _device()
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    D, B, Hq, H = case["D"], case["B"], case["Hq"], case["Hkv"]
    dt = DT[case["dtype"]]
    s = dict(case=case, D=D, B=B, Hq=Hq, H=H, dt=dt)
    s["two"] = _byte_values(dev)
    if case["op"] == "decode4":
        lens = _lengths(case)
        nb = int(np.sum(-(-lens.astype(np.int64) // B)))
        nb = nb * 10 // 9 + 2
        s["bt"] = _tables(lens, B, nb, g, dev)
        s["lens"] = torch.from_numpy(lens).to(dev)
        s["k_scale"], s["v_scale"] = 0.625, 0.75
        s["k"] = _pool4(nb, H, B, D, case["sigma"], s["k_scale"], g, dev)
        s["v"] = _pool4(nb, H, B, D, case["sigma"], s["v_scale"], g, dev)
        s["q"] = torch.randn(len(lens), Hq, D, generator=g, device=dev).to(dt)
        s["scale"] = 1.0 / math.sqrt(D)
        return s
    seq, pos, lens = _tokens(case)
    n = len(seq)
    nb = int(np.sum(-(-lens // B)))
    nb = nb * 10 // 9 + 2
    s["bt"] = _tables(lens, B, nb, g, dev)
    s["seq"] = torch.from_numpy(seq).to(dev)
    s["pos"] = torch.from_numpy(pos).to(dev)
    # the fused projection's output: queries, keys and values are views of its rows
    x = torch.randn(n, (Hq + 2 * H) * D, generator=g, device=dev).to(dt)
    s["qx"] = x[:, :Hq * D].view(n, Hq, D)
    s["kx"] = x[:, Hq * D:(Hq + H) * D].view(n, H, D)
    s["vx"] = x[:, (Hq + H) * D:].view(n, H, D)
    s["k_scale"], s["v_scale"] = (0.625, 0.75) if case["pool"] == "e2m1" else (0.0109375, 0.0125)
    s["k_st"], s["v_st"] = torch.tensor([s["k_scale"], s["v_scale"]], device=dev)
    if case["op"] == "write4":
        s["kx"], s["vx"] = s["kx"].contiguous(), s["vx"].contiguous()
    if case["rot"]:
        # the model's table of angles, computed in 64 bits once
        rot = case["rot"]
        inv = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=dev) / rot)
        a = torch.arange(int(lens.max()), dtype=torch.float64, device=dev)[:, None] * inv[None]
        s["cos_sin"] = torch.cat((a.cos(), a.sin()), -1).float()
    if case["norm"]:
        s["q_norm"] = (1 + 0.2 * torch.randn(D, generator=g, device=dev)).to(dt)
        s["k_norm"] = (1 + 0.2 * torch.randn(D, generator=g, device=dev)).to(dt)
    if case["pool"] == "e2m1":
        s["k"] = _pool4(nb, H, B, D, 1.0, s["k_scale"], g, dev)
        s["v"] = _pool4(nb, H, B, D, 1.0, s["v_scale"], g, dev)
    elif case["pool"] == "e4m3":
        for name, sc in (("k", s["k_scale"]), ("v", s["v_scale"])):
            r = torch.randn(nb, B, H, D, generator=g, device=dev) / sc
            s[name] = r.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    else:
        s["k"] = torch.randn(nb, B, H, D, generator=g, device=dev).to(dt)
        s["v"] = torch.randn(nb, B, H, D, generator=g, device=dev).to(dt)
    return s


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------

def _normed(x, w):
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * w.float()


def _rotated(x, cs, rot, interleaved):
    """x [n, heads, D], cs [n, rot] (cosines, then sines), in 32 bits."""
    h = rot // 2
    c, s = cs[:, None, :h], cs[:, None, h:]
    out = x.clone()
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        out[..., 0:rot:2], out[..., 1:rot:2] = a * c - b * s, b * c + a * s
    else:
        a, b = x[..., :h], x[..., h:rot]
        out[..., :h], out[..., h:rot] = a * c - b * s, b * c + a * s
    return out


def _plain_append(s):
    case, D, B = s["case"], s["D"], s["B"]
    q, k = s["qx"].float(), s["kx"].float()
    if case["norm"]:
        q, k = _normed(q, s["q_norm"]), _normed(k, s["k_norm"])
    if case["rot"]:
        cs = s["cos_sin"][s["pos"].long()]
        q = _rotated(q, cs, case["rot"], case["interleaved"])
        k = _rotated(k, cs, case["rot"], case["interleaved"])
    q, k, v = q.to(s["dt"]), k.to(s["dt"]), s["vx"]
    pos = s["pos"].long()
    blk, row = s["bt"][s["seq"].long(), pos // B].long(), pos % B
    if case["pool"] == "16":
        s["k"][blk, row], s["v"][blk, row] = k, v
        return {"q": q, "k": s["k"], "v": s["v"]}
    if case["pool"] == "e4m3":
        for name, x in (("k", k), ("v", v)):
            y = x.float() / s[name + "_st"]
            s[name][blk, row] = y.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        return {"q": q, "k": s["k"].view(torch.float8_e4m3fn),
                "v": s["v"].view(torch.float8_e4m3fn)}
    out = {"q": q} if case["op"] == "append" else {}
    for name, x in (("k", k), ("v", v)):
        _store4(s[name], x.float(), blk, row, s[name + "_st"], D, B)
        out[name] = _load4(s[name], blk, row, s[name + "_scale"], D, B, s["dt"], s["two"])
    return out


def _plain_decode(s):
    D, B, H, Hq = s["D"], s["B"], s["H"], s["Hq"]
    N, width = s["bt"].shape
    blk = s["bt"].clamp(min=0).long()
    T = s["lens"].long()
    t = torch.arange(width * B, device=T.device)
    live = t[None] < T[:, None]
    if s["case"]["window"]:
        live = live & (t[None] >= (T - s["case"]["window"])[:, None])

    def rows(pool):          # [N, H, width * B, D]
        codes, scales = _views4(pool, D, B)
        c = codes[blk].permute(0, 2, 1, 3, 4).reshape(N, H, width * B, D // 2)
        sc = scales[blk].permute(0, 2, 1, 3, 5, 4).reshape(N, H, width * B, D // 16)
        return _values4(c, sc, s["two"])

    q = s["q"].float().view(N, H, Hq // H, D)
    x = (q @ rows(s["k"]).transpose(-1, -2)) * (s["scale"] * s["k_scale"])
    x = torch.where(live[:, None, None], x, torch.full_like(x, -math.inf))
    m = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(m > -math.inf, m, torch.zeros_like(m)))
    o = (p @ rows(s["v"])) / p.sum(-1, keepdim=True).clamp(min=1e-30) * s["v_scale"]
    return o.view(N, Hq, D).to(s["dt"])


def _own_append(s):
    import paged_kv_cache_72_gb300 as pa
    case = s["case"]
    if "q_out" not in s:     # the step's buffers, kept by the caller
        n = s["seq"].numel()
        s["q_out"] = torch.empty(n, s["Hq"], s["D"], dtype=s["dt"], device=s["seq"].device)
        s["slots"] = torch.empty(n, dtype=torch.int64, device=s["seq"].device)
        if case["pool"] == "e2m1":
            s["k_rows"] = torch.empty(n, s["H"], s["D"], dtype=s["dt"], device=s["seq"].device)
            s["v_rows"] = torch.empty_like(s["k_rows"])
            shape = pa.pa_fp4_pool_shape(s["k"].shape[0], s["B"], s["H"], s["D"])
            s["k4"], s["v4"] = s["k"].view(shape), s["v"].view(shape)
    if case["pool"] != "e2m1":
        pa.pa_append_rope(s["qx"], s["kx"], s["vx"], s["cos_sin"], s["bt"], s["seq"], s["pos"],
                          s["k"], s["v"], interleaved=case["interleaved"], q_norm=s.get("q_norm"),
                          k_norm=s.get("k_norm"), eps=EPS, k_scale=s["k_scale"],
                          v_scale=s["v_scale"], q_out=s["q_out"])
        if case["pool"] == "16":
            return {"q": s["q_out"], "k": s["k"], "v": s["v"]}
        return {"q": s["q_out"], "k": s["k"].view(torch.float8_e4m3fn),
                "v": s["v"].view(torch.float8_e4m3fn)}
    out = {}
    if case["op"] == "append":
        pa.pa_append_rope(s["qx"], s["kx"], s["vx"], s["cos_sin"], s["bt"], s["seq"], s["pos"],
                          s["k4"], s["v4"], interleaved=case["interleaved"],
                          q_norm=s.get("q_norm"), k_norm=s.get("k_norm"), eps=EPS,
                          k_scale=s["k_scale"], v_scale=s["v_scale"], q_out=s["q_out"],
                          slot_mapping=s["slots"])
        out["q"] = s["q_out"]
    else:
        pa.pa_cache_write_fp4_mapped(s["kx"], s["vx"], s["bt"], s["seq"], s["pos"], s["k4"],
                                     s["v4"], s["k_scale"], s["v_scale"],
                                     slot_mapping=s["slots"])
    out["k"], out["v"] = pa.pa_cache_read_fp4(s["slots"], s["k4"], s["v4"], s["k_scale"],
                                              s["v_scale"], k_out=s["k_rows"], v_out=s["v_rows"])
    return out


def _own_decode(s):
    import paged_kv_cache_72_gb300 as pa
    if "out" not in s:       # the output and the workspace, kept by the caller
        shape = pa.pa_fp4_pool_shape(s["k"].shape[0], s["B"], s["H"], s["D"])
        s["k4"], s["v4"] = s["k"].view(shape), s["v"].view(shape)
        s["out"] = torch.empty_like(s["q"])
        size = pa.pa_decode_workspace_size(s["Hq"], s["H"], s["D"], s["B"], pa.PA_FP4_E2M1)
        s["workspace"] = torch.zeros(size, dtype=torch.uint8, device=s["q"].device)
    return pa.pa_decode_fp4(s["q"], s["k4"], s["v4"], s["bt"], s["lens"], s["scale"],
                            s["k_scale"], s["v_scale"], window=s["case"]["window"], out=s["out"],
                            workspace=s["workspace"])


def run(state):
    if state["case"]["op"] == "decode4":
        return _own_decode(state) if own else _plain_decode(state)
    return _own_append(state) if own else _plain_append(state)


# ---------------------------------------------------------------------------
# The definition in 64 bits
# ---------------------------------------------------------------------------

def _grid(x, bits, emin, top):
    """|x| <= top rounded to the nearest value with `bits` fraction bits and exponents from
    emin, ties to even."""
    a = x.abs().clamp(max=top)
    e = torch.floor(torch.log2(a.clamp(min=2.0 ** emin)))
    e = torch.where(torch.exp2(e) > a.clamp(min=2.0 ** emin), e - 1, e)
    step = torch.exp2(e - bits)
    return torch.copysign(torch.round(a / step) * step, x)


def _four_bit64(x, scale):
    """The values that x's 4-bit form stands for, in 64 bits."""
    g = x.double().unflatten(-1, (-1, 16))
    s = _grid(g.abs().amax(-1, keepdim=True) / (6.0 * scale), 3, -6, 448.0)
    d = s * scale
    v = _grid(g / torch.where(d > 0, d, torch.ones_like(d)), 1, 0, 6.0)
    return torch.where(d > 0, v * d, torch.zeros_like(v)).flatten(-2)


def _pool_rows64(pool, blocks, D, B):
    """code * scale16 of every row of `blocks` [n], as [n * B, H, D] in 64 bits, from the
    bytes' fields."""
    p = pool[blocks].long()                                     # [n, H, bytes]
    n, H = p.shape[:2]
    c = p[..., :B * D // 2].reshape(n, H, B, D // 2)
    nib = torch.stack((c % 16, c // 16), -1).reshape(n, H, B, D)
    e, m = (nib // 2) % 4, nib % 2
    v = torch.where(e > 0, torch.exp2((e - 1).double()) * (1 + m.double() / 2), m.double() / 2)
    v = torch.where(nib >= 8, -v, v)
    b = p[..., B * D // 2:].reshape(n, H, B // 4, D // 16, 4)
    e, m = (b // 8) % 16, (b % 8).double()
    s = torch.where(e > 0, torch.exp2((e - 7).double()) * (1 + m / 8), m * 2.0 ** -9)
    s = s.permute(0, 1, 2, 4, 3).reshape(n, H, B, D // 16, 1)
    v = (v.reshape(n, H, B, D // 16, 16) * s).reshape(n, H, B, D)
    return v.permute(0, 2, 1, 3).reshape(n * B, H, D)


def _exact_decode(s):
    D, B, H, G = s["D"], s["B"], s["H"], s["Hq"] // s["H"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=s["q"].device)
    for i, T in enumerate(s["lens"].tolist()):
        first = max(0, T - s["case"]["window"]) if s["case"]["window"] else 0
        if T == 0:
            continue
        b0 = first // B
        blocks = s["bt"][i, b0:-(-T // B)].long()
        K = _pool_rows64(s["k"], blocks, D, B)[first - b0 * B:T - b0 * B] * s["k_scale"]
        V = _pool_rows64(s["v"], blocks, D, B)[first - b0 * B:T - b0 * B] * s["v_scale"]
        for h in range(H):
            x = s["q"][i, h * G:(h + 1) * G].double() @ K[:, h].T * s["scale"]
            out[i, h * G:(h + 1) * G] = torch.softmax(x, -1) @ V[:, h]
    return out


def _exact_append(s):
    case, B, rot = s["case"], s["B"], s["case"]["rot"]
    pos = s["pos"].long()

    def placed(x, w):
        x = x.double()
        if case["norm"]:
            x = x / torch.sqrt((x * x).sum(-1, keepdim=True) / s["D"] + EPS) * w.double()
        if rot:
            cs = s["cos_sin"].double()[pos]
            turn = torch.complex(cs[:, :rot // 2], cs[:, rot // 2:])[:, None]
            head, tail = x[..., :rot], x[..., rot:]
            if case["interleaved"]:
                z = torch.view_as_complex(head.reshape(head.shape[:-1] + (-1, 2)).contiguous())
                head = torch.view_as_real(z * turn).flatten(-2)
            else:
                z = torch.complex(head[..., :rot // 2], head[..., rot // 2:]) * turn
                head = torch.cat((z.real, z.imag), -1)
            x = torch.cat((head, tail), -1)
        return x

    q, k = placed(s["qx"], s.get("q_norm")), placed(s["kx"], s.get("k_norm"))
    flat = s["bt"].long()[s["seq"].long(), pos // B] * B + pos % B
    out = {"q": q} if case["op"] == "append" else {}
    for name, x in (("k", k), ("v", s["vx"].double())):
        scale = s[name + "_scale"]
        if case["pool"] == "e2m1":      # what is stored is quantized from its 16-bit value
            out[name] = _four_bit64(x.to(s["dt"]), scale)
            continue
        if case["pool"] == "e4m3":
            pool = s[name].view(torch.float8_e4m3fn).double()
            x = _grid(x.to(s["dt"]).double() / scale, 3, -6, 448.0)
        else:
            pool = s[name].double()
        pool.view(-1, s["H"], s["D"])[flat] = x
        out[name] = pool
    return out


def exact(case, seed):
    s = prepare(case, seed)
    return _exact_decode(s) if case["op"] == "decode4" else _exact_append(s)
