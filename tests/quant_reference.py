"""Attention of chunks over quantized paged caches in 64 bits, with a bound on what a
kernel with the library's roundings may be off: a plain implementation for the tests.

The bound, per output element o = sum_t w_t V_t with w the softmax of the scores (v_scale
left out), spread = sum_t w_t |V_t - o|, n attended tokens:

* each weight is off by a relative error of at most e_w: its rounding to binary16 (2^-11),
  its score's error and ex2's (2^-22).  A score is a sum of D exact products of at most
  A = scale * sum_d |q_d K_td| in magnitude, added in fp32 in steps of 16 products (at most
  D / 16 + 1 roundings of 2^-23 A), then one fused multiply-add (2^-23 A) and the reference's
  subtraction: under 2^-19 A.  A bfloat16 query loses less than 2^-24 of its row's largest
  element where an element is below 2^-14 of that: 2^-24 A' with A' = scale * max_d |q_d| *
  sum_d |K_td|.  The sum of the weights takes the same rounded weights, so a relative error
  moves o by at most e_w * spread / (1 - e_w).
* weights below 2^-14 of a reference that is at least 2^-7 under the row's largest are
  subnormal: each is off by at most 2^-25 of units in which the largest is 2^7 or more.
* sums over tokens run in fp32, 16 products a step, each step off by 2^-23 of the sum's
  magnitude: (n / 16 + 32) 2^-23 sum_t w_t |V_t|, and so is the sum of weights, which is
  divided by.  Joining the parts of a split context costs a few 2^-22 more (in the 32).
* the result is rounded once to the output's type: half a step.
"""
import numpy as np
import torch

E2M1 = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)


def e4m3_table():
    b = torch.arange(256)
    e, m = (b // 8) % 16, (b % 8).double()
    v = torch.where(e > 0, torch.exp2((e - 7).double()) * (1 + m / 8), m * 2.0 ** -9)
    v = torch.where(b % 128 == 127, torch.full_like(v, float("nan")), v)
    return torch.where(b >= 128, -v, v)


def rows64(pool, four, blocks, H, B, D):
    """What the rows of `blocks` stand for before the tensor's scale: [len(blocks) * B, H, D]."""
    e4m3 = e4m3_table().to(pool.device)
    p = pool[blocks].long()
    if not four:
        return e4m3[p].reshape(-1, H, D)
    n = p.shape[0]
    p = p.reshape(n, H, -1)
    c = p[..., :B * D // 2].reshape(n, H, B, D // 2)
    two = torch.cat((E2M1, -E2M1)).to(pool.device)
    v = torch.stack((two[c % 16], two[c // 16]), -1).reshape(n, H, B, D // 16, 16)
    s = e4m3[p[..., B * D // 2:]].reshape(n, H, B // 4, D // 16, 4).permute(0, 1, 2, 4, 3)
    v = v * s.reshape(n, H, B, D // 16, 1)
    return v.reshape(n, H, B, D).permute(0, 2, 1, 3).reshape(n * B, H, D)


def half_step(x, dtype):
    """Half the spacing of dtype's values at |x|."""
    eps, tiny = {torch.float16: (2.0 ** -10, 2.0 ** -14),
                 torch.bfloat16: (2.0 ** -7, 2.0 ** -126)}[dtype]
    e = torch.floor(torch.log2(x.abs().clamp(min=tiny)))
    return torch.exp2(e) * eps / 2


def chunk_reference(q, k, v, four, bt, lens, start, scale, k_scale, v_scale, window=0,
                    left_out=None):
    """(out, tolerance) in 64 bits for every row of q (rows of no sequence: NaN).  left_out[i]:
    tokens of sequence i that no row attends to (blocks with bad entries)."""
    if four:
        H, B = k.shape[1], k.shape[2]
    else:
        B, H = k.shape[1], k.shape[2]
    Hq, D = q.shape[1:]
    G = Hq // H
    dev = q.device
    out = torch.full(q.shape, float("nan"), dtype=torch.float64, device=dev)
    tol = torch.zeros_like(out)
    start = [int(x) for x in start]
    for i, T in enumerate(int(x) for x in lens):
        x = q[start[i]:start[i + 1]].double()
        L = x.shape[0]
        if L == 0:
            continue
        need = -(-T // B)
        first = max(0, T - L - window + 1) if window else 0
        blocks = bt[i, first // B:need].long().clamp(min=0, max=k.shape[0] - 1)
        base = first // B * B
        K = rows64(k, four, blocks, H, B, D)[:T - base].to(dev)
        V = rows64(v, four, blocks, H, B, D)[:T - base].to(dev)
        t = torch.arange(base, T, device=dev)
        p = torch.arange(T - L, T, device=dev)
        live = t[None] <= p[:, None]
        if window:
            live &= t[None] > p[:, None] - window
        if left_out and i in left_out:
            live[:, torch.tensor([int(u) in left_out[i] for u in t], device=dev)] = False
        some = live.any(-1)
        n = live.sum(-1).double()[:, None]
        for h in range(Hq):
            Kh, Vh = K[:, h // G], V[:, h // G]
            # what nobody attends to may hold anything
            used = live.any(0)
            Kh = torch.where(used[:, None], Kh, torch.zeros_like(Kh))
            Vh = torch.where(used[:, None], Vh, torch.zeros_like(Vh))
            s = (x[:, h] @ Kh.T) * (scale * k_scale)
            s = torch.where(live, s, torch.full_like(s, -float("inf")))
            w = torch.softmax(torch.where(some[:, None], s, torch.zeros_like(s)), -1)
            w = torch.where(live, w, torch.zeros_like(w))
            o = w @ Vh
            A = torch.where(live, (x[:, h].abs() @ Kh.abs().T) * abs(scale * k_scale),
                            torch.zeros_like(s)).amax(-1, keepdim=True)
            e_w = 2.0 ** -11 * (1 + 2.0 ** -6) + 2.0 ** -19 * A + 2.0 ** -20
            if q.dtype == torch.bfloat16:
                e_w = e_w + 2.0 ** -24 * abs(scale * k_scale) * (
                    x[:, h].abs().amax(-1, keepdim=True)
                    * torch.where(live, Kh.abs().sum(-1)[None], torch.zeros_like(s)).amax(
                        -1, keepdim=True))
            spread = torch.zeros_like(o)
            far = torch.zeros_like(o)
            for d0 in range(0, D, 8):      # [L, T, 8] at a time
                away = (Vh[None, :, d0:d0 + 8] - o[:, None, d0:d0 + 8]).abs()
                spread[:, d0:d0 + 8] = (w[..., None] * away).sum(1)
                far[:, d0:d0 + 8] = (away * live[..., None]).amax(1)
            off = e_w * spread * (1 + 2.0 ** -6) + n * 2.0 ** -32 * far \
                + (n / 16 + 32) * 2.0 ** -23 * (w @ Vh.abs())
            o, off = o * v_scale, off * abs(v_scale)
            out[start[i]:start[i + 1], h] = o
            tol[start[i]:start[i + 1], h] = off + half_step(o.abs() + off, q.dtype)
    return out, tol


def quantize4(x, scale):
    """float64 [n, H, B, D] -> bytes [n, H, B * 9 D / 16] of a 4-bit pool: any codes near x do
    (the reference reads the codes)."""
    n, H, B, D = x.shape
    g = x.reshape(n, H, B, D // 16, 16) / scale
    s = (np.abs(g).max(-1) / 6.0).clip(2.0 ** -9, 448.0)
    table = e4m3_table()[:127].numpy()
    s8 = np.abs(table[None] - s.reshape(-1, 1)).argmin(-1).astype(np.uint8).reshape(s.shape)
    d = np.maximum(table[s8], 2.0 ** -9)[..., None]
    code = np.abs(np.abs(g / d)[..., None] - E2M1.numpy()).argmin(-1).astype(np.uint8)
    code |= (g < 0).astype(np.uint8) << 3
    code = code.reshape(n, H, B, D)
    packed = (code[..., 0::2] | (code[..., 1::2] << 4)).reshape(n, H, -1)
    scales = s8.reshape(n, H, B // 4, 4, D // 16).transpose(0, 1, 2, 4, 3).reshape(n, H, -1)
    return np.concatenate((packed, scales), -1)


def quantize8(x, scale):
    """float64 [n, B, H, D] -> E4M3 codes."""
    y = torch.from_numpy((x / scale).astype(np.float32)).clamp(-448, 448)
    return y.to(torch.float8_e4m3fn).view(torch.uint8).numpy()


class Chunks:
    """Pools, tables and queries of one call.  What no row attends to holds NaN codes, table
    entries before the window and past the end are -1."""

    def __init__(self, seed, four, dtype, Hq, H, D, B, new, lens, window=0, sigma=1.0,
                 q_sigma=1.0, spare=5, scales=(0.3, 0.4), device="cuda", tail_rows=0):
        rng = np.random.default_rng(seed)
        self.four, self.H, self.B, self.D, self.window = four, H, B, D, window
        new, lens = np.asarray(new, np.int64), np.asarray(lens, np.int64)
        assert (new <= lens).all()
        need = -(-lens // B)
        nb = int(need.sum()) + spare
        perm = rng.permutation(nb)
        bt = np.full((len(lens), max(1, int(need.max(initial=0)))), -1, np.int32)
        shape = (nb, H, B * 9 * D // 16) if four else (nb, B, H, D)
        pools = np.full((2,) + shape, 0x7F, np.uint8)
        at = 0
        for i, n in enumerate(need):
            rows = perm[at:at + n]
            at += n
            if n == 0 or new[i] == 0:
                continue
            first = max(0, lens[i] - new[i] - window + 1) if window else 0
            lo = first // B
            bt[i, lo:n] = rows[lo:]
            t = np.arange(n)[:, None] * B + np.arange(B)
            live = (t >= first) & (t < lens[i])
            for p, sc in zip(pools, scales):
                if four:
                    b = quantize4(sigma * rng.standard_normal((n, H, B, D)), sc)
                    dead = np.repeat((~live).reshape(n, 1, B // 4, 1, 4), H, 1)
                    dead = np.repeat(dead, D // 16, 3).reshape(n, H, -1)
                    s = b[..., B * D // 2:]
                    s[dead] = 0x7F
                else:
                    b = quantize8(sigma * rng.standard_normal((n, B, H, D)), sc)
                    b[~live] = 0x7F
                p[rows] = b
        if four:
            pools = pools.reshape(2, nb, H, B, 9 * D // 16)
        self.k, self.v = (torch.from_numpy(p).to(device) for p in pools)
        self.k_scale, self.v_scale = scales
        self.scale = float(np.float32(D ** -0.5))
        self.bt = torch.from_numpy(bt).to(device)
        self.lens = torch.from_numpy(lens.astype(np.int32)).to(device)
        self.new = new
        start = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        self.start = torch.from_numpy(start).to(device)
        q = q_sigma * rng.standard_normal((int(new.sum()) + tail_rows, Hq, D))
        self.q = torch.from_numpy(q).to(device).to(dtype)
        self.err = torch.zeros(1, dtype=torch.int32, device=device)

    def run(self, pa, **kw):
        call = pa.pa_prefill_fp4 if self.four else pa.pa_prefill_fp8
        kw.setdefault("window", self.window)
        kw.setdefault("err", self.err)
        kw.setdefault("scale", self.scale)
        return call(kw.pop("q", self.q), self.k, self.v, kw.pop("bt", self.bt),
                    kw.pop("lens", self.lens), kw.pop("start", self.start), kw.pop("scale"),
                    self.k_scale, self.v_scale, **kw)

    def reference(self, device=None, scale=None, left_out=None):
        dev = device or self.q.device
        return chunk_reference(self.q.to(dev), self.k.to(dev), self.v.to(dev), self.four,
                               self.bt.to(dev), self.lens.cpu(), self.start.cpu(),
                               self.scale if scale is None else scale, self.k_scale,
                               self.v_scale, self.window, left_out)


def assert_within(got, want, tol, what=""):
    got = got.double()
    same = (got == want) | (got.isnan() & want.isnan())
    bad = ~(same | ((got - want).abs() <= tol))
    if bool(bad.any()):
        worst = torch.where(bad, ((got - want).abs() / tol).nan_to_num(1e30),
                            torch.zeros_like(tol))
        at = np.unravel_index(int(worst.argmax()), worst.shape)
        raise AssertionError("%s%d of %d elements past the bound; at %s %r for %r, bound %r" % (
            what, int(bad.sum()), bad.numel(), tuple(int(x) for x in at), float(got[at]),
            float(want[at]), float(tol[at])))
