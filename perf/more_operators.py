"""Chunks of new tokens over quantized paged KV caches, and positions with several
axes on the way into the cache, as cases that can be timed.

Two operators:

* ``chunk``: attention of each sequence's last new tokens (one, a few that are
  verified together, a chunk of a prompt) over a paged cache of E4M3 or 4-bit
  codes, causal, with an optional sliding window.
* ``axes``: a step's queries, keys and values enter the attention as in the
  append with one position a token, but the rotation takes every frequency's
  angle from the position on that frequency's axis (time, height, width), as
  tokens of images and video have them; keys and values are stored at their
  slots of the paged pools (16-bit elements, E4M3 codes or 4-bit codes).

A 4-bit pool holds E2M1 codes (0, .5, 1, 1.5, 2, 3, 4, 6 and their negatives)
with one E4M3 scale for every 16 consecutive head_dim values of a token and one
float32 scale for the tensor: value = code * scale16 * scale.  Pools are uint8
[num_blocks][num_kv_heads][B * 9 D / 16]; the bytes of a (block, head) are the
codes [B][D / 2] (the even element in the low nibble), then the scales
[B / 4][D / 16][4], the last index being the token's position modulo 4.  An E4M3
pool is uint8 [num_blocks][B][num_kv_heads][D], value = code * scale.

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

def _chunk(name, Hq, Hkv, D, B, dtype, pool, seqs, new, lo, hi, **more):
    c = dict(name=name, op="chunk", Hq=Hq, Hkv=Hkv, D=D, B=B, dtype=dtype, pool=pool, seqs=seqs,
             new=new, lo=lo, hi=hi, ragged=False, singles=0.0, window=0, sigma=1.0, len_seed=4)
    c.update(more)
    return c


def _axes(name, Hq, Hkv, D, B, dtype, pool, seqs, new, past, **more):
    c = dict(name=name, op="axes", Hq=Hq, Hkv=Hkv, D=D, B=B, dtype=dtype, pool=pool, seqs=seqs,
             new=new, past=past, rot=D, axes=3, striped=False, interleaved=False, norm=False,
             ragged=False, len_seed=5)
    c.update(more)
    return c


def listed():
    return [
        # the tiny workload's four sequences, two new tokens each
        _chunk("chunk tiny 4-bit", 8, 8, 64, 4, "fp16", "e2m1", 4, 2, 5, 31),
        # the chunked-prefill step: 16 prompts of 512 new tokens over what they have so far
        _chunk("chunk llama3-8b 4-bit", 32, 8, 128, 16, "bf16", "e2m1", 16, 512, 0, 6144),
        # the 70B-class layer verifying four proposed tokens of 32 long contexts
        _chunk("chunk 70b verify 4-bit", 64, 8, 128, 16, "bf16", "e2m1", 32, 4, 16384, 32764),
        # a serving step: most sequences bring one token, some a chunk of their prompt
        _chunk("chunk llama3-8b mixed e4m3", 32, 8, 128, 16, "bf16", "e4m3", 64, 256, 0, 2048,
               ragged=True, singles=0.75, sigma=0.5),
        # ragged chunks without grouped heads, sliding window
        _chunk("chunk llama2-7b window e4m3", 32, 32, 128, 16, "fp16", "e4m3", 7, 277, 0, 1500,
               ragged=True, window=512),
        # the last chunk of one 32 K prompt
        _chunk("chunk 70b prompt e4m3", 64, 8, 128, 16, "bf16", "e4m3", 1, 1024, 31744, 31744),
        # own suffixes over a shared prefix's length (Qwen2-0.5B's heads)
        _chunk("chunk qwen2 suffix 4-bit", 14, 2, 64, 16, "fp16", "e2m1", 12, 300, 1800, 1800,
               ragged=True),
        # positions with axes: the smallest step
        _axes("axes tiny", 8, 8, 64, 4, "fp16", "16", 4, 1, 40),
        # prompts of text and images, heads normed
        _axes("axes llama3-8b prefill", 32, 8, 128, 16, "bf16", "16", 16, 512, 6144, norm=True),
        # ragged prompts, axes dealt out in turn, neighbours paired, into an E4M3 cache
        _axes("axes llama2-7b striped e4m3", 32, 32, 128, 16, "fp16", "e4m3", 7, 277, 1500,
              striped=True, interleaved=True, ragged=True),
        # the 70B-class layer's step into a 4-bit cache
        _axes("axes 70b 4-bit step", 64, 8, 128, 16, "bf16", "e2m1", 32, 1, 32767),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    dtype = rng.choice(("bf16", "fp16"))
    D = rng.choice((64, 128, 128))
    len_seed = rng.randrange(1 << 20)
    Hkv = rng.choice((1, 2, 3, 4, 5, 8, 8, 16, 32))
    B = rng.choice((4, 8, 16, 16, 32, 64, 256))
    if rng.random() < 0.6:
        G = rng.choice((1, 2, 3, 4, 5, 7, 8, 8, 12, 16))
        while Hkv * G > 64:
            Hkv = max(1, Hkv // 2)
        seqs = _log_int(rng, 1, 64)
        # padded scores and padded rows within the largest listed cases'
        new = _log_int(rng, 1, max(1, min(1024, 8192 // seqs)))
        most = min(32768, (64 * 1024 * 32768) // (seqs * Hkv * G * new),
                   (32 * 32768 * 8 * 128) // (seqs * Hkv * D))
        hi = _log_int(rng, 1, max(1, most - new))
        lo = rng.choice((0, hi // 2, hi))
        return dict(op="chunk", Hq=Hkv * G, Hkv=Hkv, D=D, B=B, dtype=dtype,
                    pool=rng.choice(("e4m3", "e2m1")), seqs=seqs, new=new, lo=lo, hi=hi,
                    ragged=rng.random() < 0.7, singles=rng.choice((0.0, 0.0, 0.5)),
                    window=rng.choice((0, 0, _log_int(rng, 1, 4096))),
                    sigma=rng.choice((0.5, 1.0)), len_seed=len_seed)
    seqs = _log_int(rng, 1, 64)
    new = _log_int(rng, 1, max(1, 8192 // seqs))
    past = _log_int(rng, 1, 8192)
    G = rng.choice((1, 2, 4, 7, 8))
    while Hkv > 1 and Hkv * (G + 2) * D > 48 * 128:
        Hkv //= 2
    pool = rng.choice(("16", "16", "e4m3", "e2m1"))
    past = min(past, max(1, (1 << 27) // (seqs * Hkv * D)))
    return dict(op="axes", Hq=Hkv * G, Hkv=Hkv, D=D, B=B, dtype=dtype, pool=pool, seqs=seqs,
                new=new, past=past, rot=rng.choice((D, D, D // 2, 16)),
                axes=rng.choice((2, 3, 3, 4)), striped=rng.random() < 0.4,
                interleaved=rng.random() < 0.3, norm=pool == "16" and rng.random() < 0.5,
                ragged=rng.random() < 0.7, len_seed=len_seed)


def _new_and_total(case):
    """Each sequence's new tokens and its tokens after them: plain integers, the same for every
    seed."""
    rng = np.random.default_rng(case["len_seed"])
    n = case["seqs"]
    new = np.full(n, case["new"], np.int64)
    if case["ragged"] and case["new"] > 1 and n > 1:
        new = rng.integers(1, case["new"], size=n, endpoint=True)
        new[rng.integers(n)] = case["new"]
    if case["op"] == "chunk":
        new = np.where(rng.random(n) < case["singles"], 1, new)
        past = rng.integers(case["lo"], case["hi"], size=n, endpoint=True)
    else:
        past = rng.integers(0, case["past"], size=n, endpoint=True)
    return new, past + new


def _tokens(case):
    """Sequence and position of every new token."""
    new, total = _new_and_total(case)
    seq = np.repeat(np.arange(len(new)), new)
    nth = np.arange(len(seq)) - np.repeat(np.cumsum(new) - new, new)
    return seq, (total - new)[seq] + nth


def _axis_positions(case):
    """int [axes, tokens]: every sequence is text, then a grid of patches (which share one time and
    count their rows and columns), then text that goes on from the grid's largest position."""
    seq, pos = _tokens(case)
    _, total = _new_and_total(case)
    rng = np.random.default_rng(case["len_seed"] + 1)
    n = len(total)
    start = np.minimum((total * rng.random(n)).astype(np.int64), total - 1)[seq]
    rows, cols = rng.integers(1, 40, size=n)[seq], rng.integers(1, 40, size=n)[seq]
    k = pos - start
    inside = (k >= 0) & (k < rows * cols)
    after = start + np.maximum(rows, cols) + (k - rows * cols)
    text = np.where(k < 0, pos, np.minimum(after, pos))
    grid = np.stack([start, start + k // cols, start + k % cols, start], 0)[:case["axes"]]
    if case["axes"] == 2:      # rows and columns alone
        grid = np.stack([start + k // cols, start + k % cols], 0)
    return np.where(inside[None], np.minimum(grid, total[seq][None] - 1), text[None])


def _axis_of(case):
    """The axis of every frequency: runs of frequencies (the first axis a quarter of them with
    three axes), or in turn."""
    n, axes = case["rot"] // 2, case["axes"]
    i = np.arange(n)
    if case["striped"]:
        return i % axes
    if axes == 3:
        return np.where(i < n // 4, 0, np.where(i < n // 4 + 3 * n // 8, 1, 2))
    return i * axes // n


def _row_bytes(case):
    """Bytes of one token's K or V row of one head in the pool."""
    D = case["D"]
    return {"16": 2 * D, "e4m3": D, "e2m1": 9 * D // 16}[case["pool"]]


def work(case):
    D, Hq, H = case["D"], case["Hq"], case["Hkv"]
    new, total = _new_and_total(case)
    n = int(new.sum())
    if case["op"] == "chunk":
        _, pos = _tokens(case)
        first = np.zeros_like(total)
        seen = pos + 1
        if case["window"]:
            first = np.maximum(0, total - new - case["window"] + 1)
            seen = np.minimum(seen, case["window"])
        rows = int((total - first).sum())
        blocks = int((-(-total // case["B"]) - first // case["B"]).sum())
        return {"bytes": rows * H * 2 * _row_bytes(case) + 4 * n * Hq * D + 4 * blocks
                + 8 * case["seqs"], "flops": 4 * int(seen.sum()) * Hq * D}
    at, axis = _axis_positions(case), _axis_of(case)
    angles = sum(len(np.unique(at[x])) * int((axis == x).sum()) for x in range(case["axes"]))
    bytes_ = n * (2 * Hq + 2 * H) * D * 2 + n * 2 * H * _row_bytes(case)    # q, k, v; q, K, V out
    bytes_ += n * (12 + 4 * case["axes"]) + angles * 8 + case["rot"] // 2
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


def _pool8(num_blocks, H, B, D, sigma, scale, g, dev):
    """An E4M3 pool of quantized N(0, sigma^2) values."""
    pool = torch.empty(num_blocks, B, H, D, dtype=torch.uint8, device=dev)
    step = max(1, (1 << 26) // (H * B * D))
    for b in range(0, num_blocks, step):
        r = torch.randn(min(step, num_blocks - b), B, H, D, generator=g, device=dev)
        r = (r * (sigma / scale)).clamp(-448, 448)
        pool[b:b + step] = r.to(torch.float8_e4m3fn).view(torch.uint8)
    return pool


def prepare(case, seed):
    dev = _device()
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    D, B, Hq, H = case["D"], case["B"], case["Hq"], case["Hkv"]
    dt = DT[case["dtype"]]
    s = dict(case=case, D=D, B=B, Hq=Hq, H=H, dt=dt, two=_byte_values(dev))
    s["k_scale"], s["v_scale"] = (0.625, 0.75) if case["pool"] == "e2m1" else (0.0109375, 0.0125)
    s["k_st"], s["v_st"] = torch.tensor([s["k_scale"], s["v_scale"]], device=dev)
    new, total = _new_and_total(case)
    n = int(new.sum())
    nb = int((-(-total // B)).sum()) * 10 // 9 + 2
    s["bt"] = _tables(total, B, nb, g, dev)
    if case["op"] == "chunk":
        pool = _pool4 if case["pool"] == "e2m1" else _pool8
        s["k"] = pool(nb, H, B, D, case["sigma"], s["k_scale"], g, dev)
        s["v"] = pool(nb, H, B, D, case["sigma"], s["v_scale"], g, dev)
        s["lens"] = torch.from_numpy(total.astype(np.int32)).to(dev)
        start = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        s["start"] = torch.from_numpy(start).to(dev)
        s["most"] = int(new.max())
        s["q"] = torch.randn(n, Hq, D, generator=g, device=dev).to(dt)
        s["scale"] = 1.0 / math.sqrt(D)
        return s
    seq, pos = _tokens(case)
    s["seq"] = torch.from_numpy(seq.astype(np.int32)).to(dev)
    s["pos"] = torch.from_numpy(pos.astype(np.int32)).to(dev)
    s["at"] = torch.from_numpy(_axis_positions(case).astype(np.int32)).to(dev).contiguous()
    s["axis_of"] = torch.from_numpy(_axis_of(case).astype(np.uint8)).to(dev)
    # the fused projection's output: queries, keys and values are views of its rows
    x = torch.randn(n, (Hq + 2 * H) * D, generator=g, device=dev).to(dt)
    s["qx"] = x[:, :Hq * D].view(n, Hq, D)
    s["kx"] = x[:, Hq * D:(Hq + H) * D].view(n, H, D)
    s["vx"] = x[:, (Hq + H) * D:].view(n, H, D)
    # the model's table of angles, computed in 64 bits once
    rot = case["rot"]
    inv = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=dev) / rot)
    a = torch.arange(int(total.max()), dtype=torch.float64, device=dev)[:, None] * inv[None]
    s["cos_sin"] = torch.cat((a.cos(), a.sin()), -1).float()
    if case["norm"]:
        s["q_norm"] = (1 + 0.2 * torch.randn(D, generator=g, device=dev)).to(dt)
        s["k_norm"] = (1 + 0.2 * torch.randn(D, generator=g, device=dev)).to(dt)
    if case["pool"] == "16":
        s["k"] = torch.randn(nb, B, H, D, generator=g, device=dev).to(dt)
        s["v"] = torch.randn(nb, B, H, D, generator=g, device=dev).to(dt)
    else:
        pool = _pool4 if case["pool"] == "e2m1" else _pool8
        s["k"] = pool(nb, H, B, D, 1.0, s["k_scale"], g, dev)
        s["v"] = pool(nb, H, B, D, 1.0, s["v_scale"], g, dev)
    return s


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------

def _plain_chunk(s):
    """All sequences padded to the longest chunk and the longest context."""
    case, D, B, H, Hq = s["case"], s["D"], s["B"], s["H"], s["Hq"]
    N, width = s["bt"].shape
    blk = s["bt"].clamp(min=0).long()
    T, start = s["lens"].long(), s["start"].long()
    L = start[1:] - start[:-1]
    j = torch.arange(s["most"], device=T.device)
    row = (start[:-1, None] + j[None]).clamp(max=s["q"].shape[0] - 1)     # [N, most]
    p = (T - L)[:, None] + j[None]                                        # their positions
    t = torch.arange(width * B, device=T.device)
    live = t <= p[..., None]                                              # [N, most, width * B]
    if case["window"]:
        live = live & (t > p[..., None] - case["window"])

    def rows(pool):          # [N, H, width * B, D]
        if case["pool"] == "e4m3":
            x = pool[blk].view(torch.float8_e4m3fn).float()               # [N, width, B, H, D]
            return x.permute(0, 3, 1, 2, 4).reshape(N, H, width * B, D)
        codes, scales = _views4(pool, D, B)
        c = codes[blk].permute(0, 2, 1, 3, 4).reshape(N, H, width * B, D // 2)
        sc = scales[blk].permute(0, 2, 1, 3, 5, 4).reshape(N, H, width * B, D // 16)
        return _values4(c, sc, s["two"])

    G = Hq // H
    q = s["q"].float()[row].view(N, s["most"], H, G, D).permute(0, 2, 3, 1, 4)
    q = q.reshape(N, H, G * s["most"], D)
    x = (q @ rows(s["k"]).transpose(-1, -2)) * (s["scale"] * s["k_scale"])
    x = x.view(N, H, G, s["most"], width * B)
    x = torch.where(live[:, None, None], x, -math.inf)
    x = torch.exp(x - x.amax(-1, keepdim=True))
    norm = x.sum(-1, keepdim=True)
    o = (x.view(N, H, G * s["most"], width * B) @ rows(s["v"])).view(N, H, G, s["most"], D)
    o = (o / norm * s["v_scale"]).permute(0, 3, 1, 2, 4).reshape(N, s["most"], Hq, D)
    return o[j[None] < L[:, None]].to(s["dt"])


def _normed(x, w):
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * w.float()


def _rotated(x, c, s, rot, interleaved):
    """x [n, heads, D], c and s [n, 1, rot / 2], in 32 bits."""
    h = rot // 2
    out = x.clone()
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        out[..., 0:rot:2], out[..., 1:rot:2] = a * c - b * s, b * c + a * s
    else:
        a, b = x[..., :h], x[..., h:rot]
        out[..., :h], out[..., h:rot] = a * c - b * s, b * c + a * s
    return out


def _plain_axes(s):
    case, D, B, rot = s["case"], s["D"], s["B"], s["case"]["rot"]
    q, k = s["qx"].float(), s["kx"].float()
    if case["norm"]:
        q, k = _normed(q, s["q_norm"]), _normed(k, s["k_norm"])
    at = s["at"].long()[s["axis_of"].long()].T                  # [n, rot / 2]
    i = torch.arange(rot // 2, device=at.device)
    cos, sin = s["cos_sin"][at, i][:, None], s["cos_sin"][at, i + rot // 2][:, None]
    q = _rotated(q, cos, sin, rot, case["interleaved"]).to(s["dt"])
    k = _rotated(k, cos, sin, rot, case["interleaved"]).to(s["dt"])
    v = s["vx"]
    pos = s["pos"].long()
    blk, row = s["bt"][s["seq"].long(), pos // B].long(), pos % B
    if case["pool"] == "16":
        s["k"][blk, row], s["v"][blk, row] = k, v
        return {"q": q, "k": s["k"], "v": s["v"]}
    out = {"q": q}
    for name, x in (("k", k), ("v", v)):
        if case["pool"] == "e4m3":
            y = x.float() / s[name + "_st"]
            s[name][blk, row] = y.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
            out[name] = s[name].view(torch.float8_e4m3fn)
        else:
            _store4(s[name], x.float(), blk, row, s[name + "_st"], D, B)
            out[name] = _load4(s[name], blk, row, s[name + "_scale"], D, B, s["dt"], s["two"])
    return out


def _four_bit_shape(s):
    """The 4-bit pools in the shape that the package's calls take, kept by the caller."""
    import paged_kv_cache_72_gb300 as pa
    if "k4" not in s:
        shape = pa.pa_fp4_pool_shape(s["k"].shape[0], s["B"], s["H"], s["D"])
        s["k4"], s["v4"] = s["k"].view(shape), s["v"].view(shape)
    return s["k4"], s["v4"]


def _own_chunk(s):
    import paged_kv_cache_72_gb300 as pa
    case = s["case"]
    if "out" not in s:       # the output and the workspace, kept by the caller
        s["out"] = torch.empty_like(s["q"])
        size = pa.pa_prefill_quant_workspace_size(s["Hq"], s["H"], s["D"])
        s["workspace"] = torch.zeros(size, dtype=torch.uint8, device=s["q"].device)
    more = dict(window=case["window"], out=s["out"], workspace=s["workspace"])
    if case["pool"] == "e4m3":
        return pa.pa_prefill_fp8(s["q"], s["k"], s["v"], s["bt"], s["lens"], s["start"],
                                 s["scale"], s["k_scale"], s["v_scale"], **more)
    k, v = _four_bit_shape(s)
    return pa.pa_prefill_fp4(s["q"], k, v, s["bt"], s["lens"], s["start"], s["scale"],
                             s["k_scale"], s["v_scale"], **more)


def _own_axes(s):
    import paged_kv_cache_72_gb300 as pa
    case = s["case"]
    if "q_out" not in s:     # the step's buffers, kept by the caller
        n, dev = s["seq"].numel(), s["seq"].device
        s["q_out"] = torch.empty(n, s["Hq"], s["D"], dtype=s["dt"], device=dev)
        if case["pool"] == "e2m1":
            s["slots"] = torch.empty(n, dtype=torch.int64, device=dev)
            s["k_rows"] = torch.empty(n, s["H"], s["D"], dtype=s["dt"], device=dev)
            s["v_rows"] = torch.empty_like(s["k_rows"])
    k, v = _four_bit_shape(s) if case["pool"] == "e2m1" else (s["k"], s["v"])
    pa.pa_append_rope_axes(s["qx"], s["kx"], s["vx"], s["cos_sin"], s["axis_of"], s["at"],
                           s["bt"], s["seq"], s["pos"], k, v, interleaved=case["interleaved"],
                           q_norm=s.get("q_norm"), k_norm=s.get("k_norm"), eps=EPS,
                           k_scale=s["k_scale"], v_scale=s["v_scale"], q_out=s["q_out"],
                           slot_mapping=s.get("slots"))
    if case["pool"] == "16":
        return {"q": s["q_out"], "k": s["k"], "v": s["v"]}
    if case["pool"] == "e4m3":
        return {"q": s["q_out"], "k": s["k"].view(torch.float8_e4m3fn),
                "v": s["v"].view(torch.float8_e4m3fn)}
    rows = pa.pa_cache_read_fp4(s["slots"], k, v, s["k_scale"], s["v_scale"], k_out=s["k_rows"],
                                v_out=s["v_rows"])
    return {"q": s["q_out"], "k": rows[0], "v": rows[1]}


def run(state):
    if state["case"]["op"] == "chunk":
        return _own_chunk(state) if own else _plain_chunk(state)
    return _own_axes(state) if own else _plain_axes(state)


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


def _e4m3_64(b):
    """The E4M3 values of the bytes b, from their fields, in 64 bits."""
    e, m = (b // 8) % 16, (b % 8).double()
    v = torch.where(e > 0, torch.exp2((e - 7).double()) * (1 + m / 8), m * 2.0 ** -9)
    return torch.where(b >= 128, -v, v)


def _pool_rows64(case, pool, blocks, D, B):
    """Every row of `blocks` [n] before the tensor's scale, as [n * B, H, D] in 64 bits, from
    the bytes' fields."""
    p = pool[blocks].long()
    if case["pool"] == "e4m3":
        return _e4m3_64(p).reshape(-1, p.shape[2], D)
    n, H = p.shape[:2]
    c = p[..., :B * D // 2].reshape(n, H, B, D // 2)
    nib = torch.stack((c % 16, c // 16), -1).reshape(n, H, B, D)
    e, m = (nib // 2) % 4, nib % 2
    v = torch.where(e > 0, torch.exp2((e - 1).double()) * (1 + m.double() / 2), m.double() / 2)
    v = torch.where(nib >= 8, -v, v)
    s = _e4m3_64(p[..., B * D // 2:].reshape(n, H, B // 4, D // 16, 4))
    s = s.permute(0, 1, 2, 4, 3).reshape(n, H, B, D // 16, 1)
    v = (v.reshape(n, H, B, D // 16, 16) * s).reshape(n, H, B, D)
    return v.permute(0, 2, 1, 3).reshape(n * B, H, D)


def _exact_chunk(s):
    case, D, B, H, G = s["case"], s["D"], s["B"], s["H"], s["Hq"] // s["H"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=s["q"].device)
    start = s["start"].tolist()
    for i, T in enumerate(s["lens"].tolist()):
        q = s["q"][start[i]:start[i + 1]].double()
        L = q.shape[0]
        blocks = s["bt"][i, :-(-T // B)].long()
        K = _pool_rows64(case, s["k"], blocks, D, B)[:T] * s["k_scale"]
        V = _pool_rows64(case, s["v"], blocks, D, B)[:T] * s["v_scale"]
        ahead = torch.ones(L, T, dtype=torch.bool, device=q.device).triu(T - L + 1)
        if case["window"]:
            ahead |= torch.ones_like(ahead).tril(T - L - case["window"])
        for h in range(H * G):
            x = (q[:, h] @ K[:, h // G].T * s["scale"]).masked_fill(ahead, -math.inf)
            out[start[i]:start[i + 1], h] = torch.softmax(x, -1) @ V[:, h // G]
    return out


def _exact_axes(s):
    case, B, rot = s["case"], s["B"], s["case"]["rot"]
    pos = s["pos"].long()
    table = s["cos_sin"].double()
    col = torch.arange(rot // 2, device=pos.device)
    at = torch.stack([s["at"][x].long() for x in s["axis_of"].tolist()], -1)
    turn = torch.complex(table[at, col], table[at, col + rot // 2])[:, None]

    def placed(x, w):
        x = x.double()
        if case["norm"]:
            x = x / torch.sqrt((x * x).sum(-1, keepdim=True) / s["D"] + EPS) * w.double()
        head, tail = x[..., :rot], x[..., rot:]
        if case["interleaved"]:
            z = torch.view_as_complex(head.reshape(head.shape[:-1] + (-1, 2)).contiguous())
            head = torch.view_as_real(z * turn).flatten(-2)
        else:
            z = torch.complex(head[..., :rot // 2], head[..., rot // 2:]) * turn
            head = torch.cat((z.real, z.imag), -1)
        return torch.cat((head, tail), -1)

    q, k = placed(s["qx"], s.get("q_norm")), placed(s["kx"], s.get("k_norm"))
    flat = s["bt"].long()[s["seq"].long(), pos // B] * B + pos % B
    out = {"q": q}
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
    return _exact_chunk(s) if case["op"] == "chunk" else _exact_axes(s)
