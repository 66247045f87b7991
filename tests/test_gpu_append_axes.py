"""The append with positions of several axes against the formula in 64 bits and against the
append with one position, to which it reduces bit for bit."""
import numpy as np
import pytest
import torch

import paged_kv_cache_72_gb300 as pa
from quant_reference import half_step

pytestmark = pytest.mark.gpu

F16, BF16 = torch.float16, torch.bfloat16


def axis_map(kind, rot, axes):
    n = rot // 2
    i = np.arange(n)
    if kind == "striped":
        a = i % axes
    elif kind == "runs":
        a = i * axes // n
    elif kind == "quads":       # runs that are not whole quads
        a = ((i + 2) // 4) % axes
    else:
        a = np.random.default_rng(n).integers(0, axes, size=n)
    return torch.from_numpy(a.astype(np.uint8)).cuda()


class Step:
    def __init__(self, seed, dtype, Hq, H, D, B, n, rot, axes=3, kind="runs", pool="16", seqs=3,
                 max_pos=500, norm=False, length=200):
        g = torch.Generator(device="cuda").manual_seed(seed)
        rng = np.random.default_rng(seed)
        self.dtype, self.D, self.B, self.H, self.Hq, self.rot = dtype, D, B, H, Hq, rot
        x = torch.randn(n, (Hq + 2 * H) * D, generator=g, device="cuda").to(dtype)
        self.q = x[:, :Hq * D].view(n, Hq, D)
        self.k = x[:, Hq * D:(Hq + H) * D].view(n, H, D)
        self.v = x[:, (Hq + H) * D:].view(n, H, D)
        self.axis_of = axis_map(kind, rot, axes)
        self.rot_pos = torch.from_numpy(
            rng.integers(0, max_pos, size=(axes, n)).astype(np.int32)).cuda()
        a = torch.rand(max_pos, rot // 2, generator=g, device="cuda", dtype=torch.float64) * 6.28
        self.cos_sin = torch.cat((a.cos(), a.sin()), -1).float()
        where = rng.permutation(seqs * length)[:n]
        self.seq = torch.from_numpy((where // length).astype(np.int32)).cuda()
        self.pos = torch.from_numpy((where % length).astype(np.int32)).cuda()
        width = -(-length // B)
        nb = seqs * width + 3
        self.nb = nb
        self.bt = torch.from_numpy(
            rng.permutation(nb)[:seqs * width].reshape(seqs, width).astype(np.int32)).cuda()
        shape = {"16": (nb, B, H, D), "e4m3": (nb, B, H, D),
                 "e2m1": pa.pa_fp4_pool_shape(nb, B, H, D)}[pool]
        kind16 = dtype if pool == "16" else torch.uint8
        self.pools = [torch.zeros(shape, dtype=kind16, device="cuda") for _ in range(2)]
        self.norms = {}
        if norm:
            self.norms = {m: (1 + 0.2 * torch.randn(D, generator=g, device="cuda")).to(dtype)
                          for m in ("q_norm", "k_norm")}
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")

    def run(self, **kw):
        kw = dict(k_scale=0.3, v_scale=0.4, err=self.err, **self.norms) | kw
        return pa.pa_append_rope_axes(self.q, self.k, self.v, self.cos_sin, self.axis_of,
                                      self.rot_pos, self.bt, self.seq, self.pos, *self.pools,
                                      **kw)

    def turned(self, x, w, interleaved):
        """The row's value in 64 bits, and a bound on what fp32 steps may be off."""
        x = x.double()
        if w is not None:
            x = x / torch.sqrt(x.square().mean(-1, keepdim=True) + 1e-6) * w.double()
        h = self.rot // 2
        at = self.rot_pos.long()[self.axis_of.long()].T
        i = torch.arange(h, device="cuda")
        c = self.cos_sin.double()[at, i][:, None]
        s = self.cos_sin.double()[at, i + h][:, None]
        out, mag = x.clone(), x.abs()
        if interleaved:
            sl = slice(0, self.rot, 2), slice(1, self.rot, 2)
        else:
            sl = slice(0, h), slice(h, self.rot)
        a, b = x[..., sl[0]], x[..., sl[1]]
        out[..., sl[0]], out[..., sl[1]] = a * c - b * s, b * c + a * s
        mag[..., sl[0]], mag[..., sl[1]] = (a * c).abs() + (b * s).abs(), (b * c).abs() + (a * s).abs()
        # fp32: a product each and a sum; with a norm the mean of D squares (D / 8 + 6 roundings,
        # halved by the root), the root, its product and the weight's with the angle
        steps = 2 if w is None else 2 + 3 + (self.D / 8 + 6) / 2 + 4
        return out, steps * 2.0 ** -24 * mag + half_step(out.abs() * (1 + 2.0 ** -18) + mag * 2.0 ** -20, self.dtype)

    def slots(self):
        p = self.pos.long()
        return self.bt.long()[self.seq.long(), p // self.B] * self.B + p % self.B


def check16(st, interleaved=False):
    out = st.run(interleaved=interleaved)
    assert pa.pa_get_error(st.err) == 0
    want, tol = st.turned(st.q, st.norms.get("q_norm"), interleaved)
    assert bool(((out.double() - want).abs() <= tol).all())
    want, tol = st.turned(st.k, st.norms.get("k_norm"), interleaved)
    k, v = (p.view(-1, st.H, st.D) for p in st.pools)
    slots = st.slots()
    assert bool(((k[slots].double() - want).abs() <= tol).all())
    assert torch.equal(v[slots], st.v)
    rest = torch.ones(k.shape[0], dtype=torch.bool, device="cuda")
    rest[slots] = False
    assert bool((k[rest] == 0).all()) and bool((v[rest] == 0).all())


@pytest.mark.parametrize("dtype", [F16, BF16], ids=["fp16", "bf16"])
@pytest.mark.parametrize("D,rot", [(64, 64), (64, 16), (128, 128), (128, 64), (128, 48)])
@pytest.mark.parametrize("kind", ["runs", "striped", "quads", "any"])
@pytest.mark.parametrize("interleaved", [False, True])
def test_formula(dtype, D, rot, kind, interleaved):
    check16(Step(1, dtype, 6, 2, D, 16, 37, rot, kind=kind), interleaved)


@pytest.mark.parametrize("axes", [1, 2, 3, 4])
@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("n", [1, 2, 300])
def test_axes_norms_and_counts(axes, norm, n):
    check16(Step(2, BF16, 16, 2, 128, 8, n, 128, axes=axes, kind="any", norm=norm))
    check16(Step(3, F16, 3, 3, 64, 4, n, 32, axes=axes, kind="striped", norm=norm), True)


@pytest.mark.parametrize("pool", ["16", "e4m3", "e2m1"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("norm", [False, True])
def test_equal_positions_are_the_append(pool, interleaved, norm):
    """rot_pos = token_pos on every axis: pa_append_rope bit for bit, in every pool."""
    st = Step(4, BF16, 8, 2, 128, 16, 90, 64, axes=3, kind="any", pool=pool, norm=norm)
    st.rot_pos[:] = st.pos[None]
    out = st.run(interleaved=interleaved)
    mine = [p.clone() for p in st.pools]
    for p in st.pools:
        p.zero_()
    one = pa.pa_append_rope(st.q, st.k, st.v, st.cos_sin, st.bt, st.seq, st.pos, *st.pools,
                            interleaved=interleaved, k_scale=0.3, v_scale=0.4, **st.norms)
    assert torch.equal(out, one)
    for a, b in zip(mine, st.pools):
        assert torch.equal(a, b)


@pytest.mark.parametrize("pool", ["e4m3", "e2m1"])
def test_quantized_pools_hold_the_rotated_rows(pool):
    """What a quantized pool ends with is its own write of the rotated 16-bit keys."""
    st = Step(5, F16, 4, 2, 64, 16, 70, 64, kind="striped", pool=pool)
    st.run()
    plain = Step(5, F16, 4, 2, 64, 16, 70, 64, kind="striped")
    plain.run()
    slots = st.slots()
    keys = plain.pools[0].view(-1, 2, 64)[slots].contiguous()
    pools = [torch.zeros_like(p) for p in st.pools]
    write = pa.pa_cache_write_fp8 if pool == "e4m3" else pa.pa_cache_write_fp4
    write(keys, st.v.contiguous(), slots, *pools, 0.3, 0.4)
    for a, b in zip(pools, st.pools):
        assert torch.equal(a, b)


def test_cache_positions_past_the_table_of_angles():
    """token_pos only places the token: it may pass max_pos."""
    check16(Step(6, BF16, 4, 2, 128, 16, 50, 128, max_pos=7))


def test_bad_positions_and_padding():
    st = Step(7, BF16, 4, 2, 128, 16, 12, 128)
    good = Step(7, BF16, 4, 2, 128, 16, 12, 128)
    good.run()
    st.rot_pos[0, 1] = -1
    st.rot_pos[2, 4] = 500
    st.rot_pos[1, 5] = 2 ** 31 - 1
    st.seq[7] = -1
    slots = torch.full((12,), 99, dtype=torch.int64, device="cuda")
    out = torch.full_like(st.q, 5.0).contiguous()
    st.run(q_out=out, slot_mapping=slots)
    assert pa.pa_get_error(st.err) == pa.PA_DEVERR_POSITION
    dead = torch.tensor([1, 4, 5, 7], device="cuda")
    assert bool((slots[dead] == -1).all()) and bool((out[dead] == 5.0).all())
    live = torch.tensor([i for i in range(12) if i not in (1, 4, 5, 7)], device="cuda")
    assert torch.equal(slots[live], good.slots()[live])
    k, kg = st.pools[0].view(-1, 2, 128), good.pools[0].view(-1, 2, 128)
    assert torch.equal(k[good.slots()[live]], kg[good.slots()[live]])
    assert bool((k[good.slots()[dead]] == 0).all())
    # padding alone is no error, whatever its positions hold
    st.rot_pos[:] = 0
    st.seq[7] = -1
    st.rot_pos[0, 7] = -3
    st.run()
    assert pa.pa_get_error(st.err) == 0


def test_bad_axis_map():
    st = Step(8, BF16, 4, 2, 128, 16, 12, 128, axes=3)
    st.axis_of[63] = 3
    out = torch.full_like(st.q, 5.0).contiguous()
    st.run(q_out=out)
    assert pa.pa_get_error(st.err) == pa.PA_DEVERR_POSITION
    assert bool((out == 5.0).all()) and bool((st.pools[0] == 0).all())


def test_captured_and_replayed():
    st = Step(9, BF16, 4, 2, 128, 16, 40, 128)
    out = torch.zeros(40, 4, 128, dtype=BF16, device="cuda")
    st.run(q_out=out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        st.run(q_out=out)
    st.rot_pos.copy_(torch.randint(0, 500, (3, 40), device="cuda", dtype=torch.int32))
    out.zero_()
    graph.replay()
    want, tol = st.turned(st.q, None, False)
    assert bool(((out.double() - want).abs() <= tol).all())


@pytest.mark.parametrize("pool", ["e4m3", "e2m1"])
@pytest.mark.parametrize("dtype", [F16, BF16], ids=["fp16", "bf16"])
def test_append_then_chunk(pool, dtype):
    """A step as a model runs it: the appends of two chunks of text and patches, then the
    attention of the second over the cache that both wrote."""
    from quant_reference import assert_within, chunk_reference
    H, Hq, D, B, T, L = 2, 8, 128, 16, 150, 60
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(T, (Hq + 2 * H) * D, generator=g, device="cuda").to(dtype)
    q, k, v = (x[:, :Hq * D].view(T, Hq, D), x[:, Hq * D:(Hq + H) * D].view(T, H, D),
               x[:, (Hq + H) * D:].view(T, H, D))
    a = torch.arange(T, dtype=torch.float64, device="cuda")[:, None] * 10000.0 ** (
        -torch.arange(0, D, 2, dtype=torch.float64, device="cuda") / D)
    cos_sin = torch.cat((a.cos(), a.sin()), -1).float()
    pos = torch.arange(T, device="cuda", dtype=torch.int32)
    patch = (pos - 20).clamp(min=0)
    rot_pos = torch.stack((pos.clamp(max=20), pos.clamp(max=20) + patch // 12,
                           pos.clamp(max=20) + patch % 12)).int().contiguous()
    nb = -(-T // B) + 2
    bt = torch.randperm(nb, generator=torch.Generator().manual_seed(1))[:nb - 2].int().cuda()[None]
    four = pool == "e2m1"
    shape = pa.pa_fp4_pool_shape(nb, B, H, D) if four else (nb, B, H, D)
    pools = [torch.zeros(shape, dtype=torch.uint8, device="cuda") for _ in range(2)]
    axis_of = axis_map("striped", D, 3)
    outs = []
    for at, n in ((0, T - L), (T - L, L)):
        s = slice(at, at + n)
        outs.append(pa.pa_append_rope_axes(
            q[s], k[s], v[s], cos_sin, axis_of, rot_pos[:, s].contiguous(), bt,
            torch.zeros(n, dtype=torch.int32, device="cuda"), pos[s], *pools, k_scale=0.02,
            v_scale=0.03))
    call = pa.pa_prefill_fp4 if four else pa.pa_prefill_fp8
    lens = torch.tensor([T], dtype=torch.int32, device="cuda")
    start = torch.tensor([0, L], dtype=torch.int32, device="cuda")
    out = call(outs[1], *pools, bt, lens, start, D ** -0.5, 0.02, 0.03)
    want, tol = chunk_reference(outs[1], *pools, four, bt, lens, start, D ** -0.5, 0.02, 0.03)
    assert_within(out, want, tol)
