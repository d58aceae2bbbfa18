"""GPU parity of the gated delta rule's operators (through the binding and the
C ABI) against float64 token loops.

Tolerances, in half steps of the types.  A float32 state: one token's write
rounds two sums of K products and the update, about 2 sqrt(K) + 6 half steps
(2^-24) of the state, 30 at K = 128; earlier tokens' errors are damped by the
decay and by I - b k k^T (a contraction), so they add like a random walk over
at most some 30 tokens: 30 sqrt(30) half steps = 1e-5 of the largest value.  A
float32 y adds a sum of K products: the same bound.  A bfloat16 y adds its
rounding, 2^-8 of its value, and, where the products with the state ran on
16-bit operands (11 bits, 2^-11 for each of two operands) of sums that cancel
by up to 4, 2^-8 of the largest value in all."""
import numpy as np
import pytest
import torch

from oracle import gdr as O
from selective_state_space_28_b200 import inputs as I

pytestmark = pytest.mark.gpu

TOL = 1e-5


def _ops():
    from selective_state_space_28_b200 import ops
    return ops


def _np(t):
    return t.detach().double().cpu().numpy()


def _close(got, ref, what, rel=TOL):
    """Within rel of the largest value, and for bfloat16 within a rounding of
    each value and 2^-8 of the largest."""
    rounding = 2.0 ** -8 if got.dtype == torch.bfloat16 else 0.0
    if rounding:
        rel = 2.0 ** -8
    got = _np(got)
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    assert np.isfinite(got).all(), what
    if ref.size:
        over = np.abs(got - ref) - rounding * np.abs(ref)
        assert over.max() <= rel * np.abs(ref).max() + 1e-30, "%s: %.3e over, max %.3e" % (
            what, over.max(), np.abs(ref).max())


def _dev(d):
    return {k: None if x is None else x.cuda() for k, x in d.items()}


def _scan(d, **kw):
    return _ops().gdr_chunk_scan_fwd(d["q"], d["k"], d["v"], d["dt"], d["A"], d["beta"],
                                     dt_bias=d["dt_bias"], h0=d["h0"], **kw)


def _ref(d, **kw):
    kw.setdefault("scale", d["k"].shape[-1] ** -0.5)
    return O.gdr_scan(d["q"], d["k"], d["v"], d["dt"], d["A"], d["beta"], d["dt_bias"], d["h0"], **kw)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("L", [1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 300])
def test_scan_lengths(cuda_ok, L, io):
    d = I.gdr_inputs(2, L, 2, 4, 128, 128, io=io, seed=L, h0=L % 2 == 0)
    y, h = _scan(_dev(d))
    ry, rh, _ = _ref(d)
    _close(y, ry, "y")
    _close(h, rh, "h_last")


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("hk,h,K,V", [(1, 1, 64, 64), (2, 6, 64, 128), (3, 3, 128, 64), (1, 2, 128, 96),
                                      (1, 2, 128, 256), (2, 2, 128, 200), (1, 2, 32, 40), (1, 1, 96, 33),
                                      (1, 3, 20, 5), (2, 2, 256, 64), (1, 1, 1, 1), (1, 2, 129, 130),
                                      (1, 1, 72, 7), (1, 2, 40, 128)])
def test_scan_heads(cuda_ok, hk, h, K, V, io):
    d = I.gdr_inputs(2, 140, hk, h, K, V, io=io, seed=K + V, h0=True)
    y, hl = _scan(_dev(d))
    ry, rh, _ = _ref(d)
    _close(y, ry, "y")
    _close(hl, rh, "h_last")


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("flags", [0, 1, 8, 16, 17, 25])
def test_scan_flags(cuda_ok, flags, io):
    d = I.gdr_inputs(1, 150, 1, 2, 64, 64, io=io, seed=flags)
    if not flags & 1:  # steps as they are: not negative
        d["dt"], d["dt_bias"] = d["dt"].abs() * 0.1, None
    if not flags & 8:
        d["beta"] = d["beta"].float().sigmoid().to(d["beta"].dtype)
    if not flags & 16:  # keys of length below 1, as a rule that is not normalised needs
        d["k"] = (d["k"].float() * 0.1).to(d["k"].dtype)
    y, h = _scan(_dev(d), flags=flags, scale=0.7)
    ry, rh, _ = _ref(d, flags=flags, scale=0.7)
    _close(y, ry, "y")
    _close(h, rh, "h_last")


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_scan_without_decay(cuda_ok, io):
    d = I.gdr_inputs(1, 200, 1, 2, 128, 128, io=io, seed=3, h0=True)
    d["dt"] = None
    y, h = _scan(_dev(d))
    ry, rh, _ = _ref(d)
    _close(y, ry, "y")
    _close(h, rh, "h_last")


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_scan_scales_of_values(cuda_ok, io):
    """Very large and very small values, keys and states keep their digits."""
    for vs, ks, hs in ((1e4, 1.0, 1.0), (1e-6, 1.0, 1e-6), (1e20, 1e-3, 1e15), (1.0, 1e4, 1e6), (1e-12, 30.0, 0.0)):
        d = I.gdr_inputs(1, 130, 1, 2, 128, 128, io=io, seed=9, h0=True)
        d["v"] = (d["v"].float() * vs).to(d["v"].dtype)
        d["k"] = (d["k"].float() * ks).to(d["k"].dtype)
        d["q"] = (d["q"].float() * ks).to(d["q"].dtype)
        d["h0"] = d["h0"] * hs
        y, h = _scan(_dev(d))
        ry, rh, _ = _ref(d)
        _close(y, ry, "y %g %g %g" % (vs, ks, hs))
        _close(h, rh, "h_last %g %g %g" % (vs, ks, hs))


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_scan_extreme_gates(cuda_ok, io):
    """Decays from none to total, write strengths 0 and 1, in one sequence."""
    d = I.gdr_inputs(1, 150, 1, 2, 64, 64, io=io, seed=4, h0=True)
    d["A"] = torch.tensor([-36316.0, -4e-4])
    d["dt"][:, 20:30] = -float("inf")   # no decay at all
    d["dt"][:, 50] = 30.0               # the state is gone
    d["beta"][:, 60:70] = -float("inf")  # nothing written
    d["beta"][:, 80:90] = 100.0
    y, h = _scan(_dev(d))
    ry, rh, _ = _ref(d)
    _close(y, ry, "y")
    _close(h, rh, "h_last")


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_scan_equal_keys(cuda_ok, io):
    """Keys that are all the same, written at full strength: the worst
    conditioned system within a chunk."""
    d = I.gdr_inputs(1, 130, 1, 2, 64, 64, io=io, seed=5)
    d["k"][:] = d["k"][:, :1]
    d["beta"][:] = 12.0
    y, h = _scan(_dev(d))
    ry, rh, _ = _ref(d)
    _close(y, ry, "y")
    _close(h, rh, "h_last")


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_scan_zero_rows(cuda_ok, io):
    """Keys, queries and values that are zero: nothing to normalise by."""
    d = I.gdr_inputs(1, 100, 1, 1, 64, 64, io=io, seed=6, h0=True)
    for x in ("q", "k", "v"):
        d[x][:, 10:20] = 0
    d["k"][:, 64:] = 0
    y, h = _scan(_dev(d))
    ry, rh, _ = _ref(d)
    _close(y, ry, "y")
    _close(h, rh, "h_last")


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_scan_split_and_carry(cuda_ok, io):
    """A prompt cut in two, its state handed on in place, is the prompt."""
    d = I.gdr_inputs(2, 201, 1, 2, 128, 128, io=io, seed=8, h0=True)
    ry, rh, _ = _ref(d)
    g = _dev(d)
    h = g["h0"]
    ys = []
    for s in (slice(0, 70), slice(70, 201)):
        part = {x: (g[x][:, s] if x in ("q", "k", "v", "dt", "beta") else g[x]) for x in g}
        part["h0"] = h
        y, out = _scan(part, h_last=h)
        assert out is h
        ys.append(y)
    _close(torch.cat(ys, 1), ry, "y")
    _close(h, rh, "h_last")


@pytest.mark.parametrize("n,L,hk,h,K,V", [(1, 3000, 1, 2, 128, 128), (2, 2049, 1, 1, 64, 96),
                                          (1, 4111, 1, 1, 128, 200), (3, 1500, 1, 2, 40, 64),
                                          (1, 2500, 2, 6, 128, 64)])
def test_scan_few_long(cuda_ok, n, L, hk, h, K, V):
    """Few long sequences, cut into segments that run side by side."""
    d = I.gdr_inputs(n, L, hk, h, K, V, io="bf16", seed=L, h0=L % 2 == 0)
    d["A"] = d["A"] * torch.logspace(-4, 0, h)  # long memories among them
    y, hl = _scan(_dev(d))
    ry, rh, _ = _ref(d)
    _close(y, ry, "y")
    _close(hl, rh, "h_last")


@pytest.mark.parametrize("packed", [False, True])
def test_scan_many_chunks_of_shared_keys(cuda_ok, packed):
    """Chunks enough that the heads that share keys are prepared together."""
    n, L, hk, h, K, V = 60, 970, 2, 6, 64, 64
    d = I.gdr_inputs(n, L, hk, h, K, V, io="bf16", seed=7, h0=True)
    g = _dev(d)
    if packed:
        cu = torch.arange(0, n * L + 1, L, dtype=torch.int32, device="cuda")
        y, hl = _scan({k: x.flatten(0, 1)[None] if k in ("q", "k", "v", "dt", "beta") else x for k, x in g.items()},
                      cu_seqlens=cu)
        y = y.reshape(n, L, h, V)
    else:
        y, hl = _scan(g)
    some = [0, 33, 59]
    part = {k: x[some] if k not in ("A", "dt_bias") else x for k, x in d.items()}
    ry, rh, _ = _ref(part)
    _close(y[some], ry, "y")
    _close(hl[some], rh, "h_last")


def test_scan_segments_in_a_graph(cuda_ok):
    """All launches of a cut sequence, captured and replayed on new inputs, and
    two such calls at once on streams of their own: the same bits."""
    ops = _ops()
    d = _dev(I.gdr_inputs(1, 2500, 1, 2, 128, 128, seed=13, h0=True))
    y0, h0 = _scan(d)
    ops.check_every_call(False)
    try:
        e = {x: d[x].clone() for x in d}
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            yg, hg = _scan(e)
        for seed in (14, 13):
            new = _dev(I.gdr_inputs(1, 2500, 1, 2, 128, 128, seed=seed, h0=True))
            for x in e:
                e[x].copy_(new[x])
            graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(yg, y0) and torch.equal(hg, h0)
        streams = [torch.cuda.Stream() for _ in range(3)]
        outs = [_scan(d, stream=s) for s in streams for _ in range(3)]
        torch.cuda.synchronize()
        assert all(torch.equal(y, y0) and torch.equal(h, h0) for y, h in outs)
    finally:
        ops.check_every_call(True)


def test_scan_few_long_packed(cuda_ok):
    """The same, packed: segments of very different lengths, some of them and
    one sequence empty, states updated in place, one sequence skipped."""
    lengths, hk, h, K, V = [2500, 1, 0, 130, 700], 1, 1, 128, 64
    d = I.gdr_inputs(1, sum(lengths), hk, h, K, V, io="bf16", seed=5)
    g = _dev(d)
    cache = 0.3 * torch.randn(6, h, K, V, device="cuda")
    before = cache.clone()
    slots = torch.tensor([5, 0, 2, 1, -1], dtype=torch.int32, device="cuda")
    cu = torch.tensor([0] + lengths, device="cuda").cumsum(0).to(torch.int32)
    y = torch.full((1, sum(lengths), h, V), 7.0, dtype=torch.bfloat16, device="cuda")
    g["h0"] = cache
    for _ in range(2):
        cache.copy_(before)
        _scan(g, cu_seqlens=cu, slots=slots, h_last=cache, y=y)
    for i, (slot, length) in enumerate(zip(slots.tolist(), lengths)):
        if slot < 0 or length == 0:
            continue
        s = slice(sum(lengths[:i]), sum(lengths[:i + 1]))
        part = {x: d[x][:, s] for x in ("q", "k", "v", "dt", "beta")}
        ry, rh, _ = O.gdr_scan(part["q"], part["k"], part["v"], part["dt"], d["A"], part["beta"], d["dt_bias"],
                               before[slot][None], scale=K ** -0.5)
        _close(y[:, s], ry, "y %d" % i)
        _close(cache[slot][None], rh, "state %d" % i)
    assert torch.equal(cache[[2, 3, 4]], before[[2, 3, 4]])
    assert (y[:, sum(lengths[:4]):] == 7).all()


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("K,V", [(128, 128), (64, 96), (48, 20)])
def test_scan_packed_slots(cuda_ok, K, V, io):
    """Sequences of many lengths, an empty and a skipped one among them, from
    slices of one projection, states anywhere in a cache; rows and states of
    no sequence, full of NaN, neither read nor written."""
    lengths, hk, h = [5, 64, 0, 200, 1, 65, 130], 1, 2
    total, n = sum(lengths), len(lengths)
    d = I.gdr_inputs(1, total + 9, hk, h, K, V, io=io, seed=11)
    g = _dev(d)
    qkv = torch.cat([g[x].flatten(2) for x in ("q", "k", "v")] + [g["v"].new_zeros(1, total + 9, 8)], -1)
    qkv[:, total:] = float("nan")
    q, k, v, _ = qkv.split([hk * K, hk * K, h * V, 8], -1)
    q, k, v = q.unflatten(-1, (hk, K)), k.unflatten(-1, (hk, K)), v.unflatten(-1, (h, V))
    ba = torch.cat([g["beta"], g["dt"]], -1)
    ba[:, total:] = float("nan")
    beta, dt = ba.split([h, h], -1)
    cache = 0.3 * torch.randn(n + 4, h, K, V, device="cuda")
    slots = torch.tensor([3, 0, 7, 10, 4, -1, 9], dtype=torch.int32, device="cuda")
    cache[[1, 2, 5, 6, 8]] = float("nan")
    before = cache.clone()
    skipped = sum(lengths[:5])
    qkv[:, skipped:skipped + 65] = float("nan")  # the skipped sequence
    cu = torch.tensor([0] + lengths, device="cuda").cumsum(0).to(torch.int32)
    y = torch.full((1, total + 9, h, V), 7.0, dtype=v.dtype, device="cuda")
    y2, out = _ops().gdr_chunk_scan_fwd(q, k, v, dt, g["A"], beta, dt_bias=g["dt_bias"], h0=cache,
                                        cu_seqlens=cu, slots=slots, h_last=cache, y=y)
    assert y2 is y and out is cache
    assert (y[:, total:] == 7).all() and (y[:, skipped:skipped + 65] == 7).all()
    for i, (slot, length) in enumerate(zip(slots.tolist(), lengths)):
        if slot < 0:
            continue
        s = slice(sum(lengths[:i]), sum(lengths[:i + 1]))
        part = {x: d[x][:, s] for x in ("q", "k", "v", "dt", "beta")}
        ry, rh, _ = O.gdr_scan(part["q"], part["k"], part["v"], part["dt"], d["A"], part["beta"], d["dt_bias"],
                               before[slot][None], scale=K ** -0.5)
        _close(y[:, s], ry, "y %d" % i)
        _close(cache[slot][None], rh, "state %d" % i)
    assert torch.equal(cache[2], before[2]) or torch.isnan(cache[2]).all()
    assert torch.equal(cache[7], before[7])  # the empty sequence


def test_scan_bad_bounds_are_empty_sequences(cuda_ok):
    """Bounds out of order or out of the buffer, and slots beyond the cache:
    nothing is read or written for them."""
    d = _dev(I.gdr_inputs(1, 100, 1, 1, 64, 64, seed=12))
    cu = torch.tensor([0, 20, 10, 300, 40, 60, 100], dtype=torch.int32, device="cuda")
    slots = torch.tensor([0, 1, 2, 3, 99, 4], dtype=torch.int32, device="cuda")
    cache = torch.zeros(5, 1, 64, 64, device="cuda")
    y = torch.full((1, 100, 1, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    d["h0"] = cache
    _scan(d, cu_seqlens=cu, slots=slots, h_last=cache, y=y)
    torch.cuda.synchronize()
    assert (y[:, 20:60] == 7).all() and (y[:, :20] != 7).any() and (y[:, 60:] != 7).any()
    assert (cache[1:4] == 0).all() and (cache[0] != 0).any() and (cache[4] != 0).any()


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_bounds_out_of_order_leave_the_others(cuda_ok, io):
    """A sequence of several chunks whose successors' bounds go back is the
    sequence all the same, in the scan and in the convolution."""
    n, hk, h, K, V = 500, 1, 1, 64, 64
    d = I.gdr_inputs(1, n, hk, h, K, V, io=io, seed=14)
    bounds = [0, 400, 10, 5, 400, 500]
    cu = torch.tensor(bounds, dtype=torch.int32, device="cuda")
    slots = torch.tensor([3, 0, 1, -1, 2], dtype=torch.int32, device="cuda")  # (5 .. 400 is skipped)
    cache = torch.zeros(4, h, K, V, device="cuda")
    g = _dev(d)
    g["h0"] = cache
    y, _ = _scan(g, cu_seqlens=cu, slots=slots, h_last=cache)
    x, w = torch.randn(n, 64), torch.randn(64, 4)
    u, _ = _ops().ssm_conv1d_packed_fwd(x.cuda(), w.cuda(), cu_seqlens=cu, slots=slots)
    for a, b, slot in ((0, 400, 3), (400, 500, 2)):
        part = {k: d[k][:, a:b] for k in ("q", "k", "v", "dt", "beta")}
        ry, rh, _ = O.gdr_scan(part["q"], part["k"], part["v"], part["dt"], d["A"], part["beta"], d["dt_bias"],
                               None, scale=K ** -0.5)
        _close(y[:, a:b], ry, "y")
        _close(cache[slot][None], rh, "state")
        _close(u[a:b], O.conv1d_packed(x[a:b], w, None, None, [b - a])[0], "u")


def test_scan_no_tokens(cuda_ok):
    d = _dev(I.gdr_inputs(2, 0, 1, 2, 128, 128, seed=1, h0=True))
    y, h = _scan(d)
    assert y.shape == (2, 0, 2, 128) and torch.equal(h, d["h0"])
    d["h0"] = None
    assert (_scan(d)[1] == 0).all()
    e = _dev(I.gdr_inputs(0, 5, 1, 2, 128, 128, seed=1))
    y, h = _scan(e)
    assert y.shape[0] == 0 and h.shape[0] == 0


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_scan_other_stream_and_graph(cuda_ok, io):
    """On a stream of its own, from slices that must be copied, and replayed
    from a graph on new inputs: the same bits."""
    ops = _ops()
    d = _dev(I.gdr_inputs(2, 90, 2, 2, 64, 64, io=io, seed=13, h0=True))
    y0, h0 = _scan(d)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    odd = dict(d)
    wide = torch.zeros(2, 90, 2, 65, dtype=d["q"].dtype, device="cuda")
    wide[..., 1:] = d["q"]
    odd["q"] = wide[..., 1:]
    torch.cuda.synchronize()
    y1, h1 = _scan(odd, stream=side)
    y2, h2 = _scan(odd, stream=side.cuda_stream)
    side.synchronize()
    for y, h in ((y1, h1), (y2, h2)):
        assert torch.equal(y, y0) and torch.equal(h, h0)
    ops.check_every_call(False)  # a status read cannot be captured
    try:
        e = {x: None if d[x] is None else d[x].clone() for x in d}
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            yg, hg = _scan(e)
        for seed in (14, 13):
            new = _dev(I.gdr_inputs(2, 90, 2, 2, 64, 64, io=io, seed=seed, h0=True))
            for x in e:
                e[x].copy_(new[x])
            graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(yg, y0) and torch.equal(hg, h0)
    finally:
        ops.check_every_call(True)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("hk,h,K,V", [(1, 1, 64, 64), (4, 8, 128, 128), (3, 9, 64, 96), (1, 2, 128, 256),
                                      (1, 2, 33, 7), (2, 2, 256, 130), (1, 1, 1, 1), (1, 1, 256, 128),
                                      (1, 1, 17, 300), (1, 2, 96, 36)])
def test_step(cuda_ok, hk, h, K, V, io):
    b = 5
    d = I.gdr_inputs(b, 1, hk, h, K, V, io=io, seed=K, h0=True)
    ry, rh, _ = _ref(d)
    g = _dev(d)
    state = g["h0"].clone()
    y = _ops().gdr_scan_step(state, g["q"][:, 0], g["k"][:, 0], g["v"][:, 0], g["dt"][:, 0], g["A"],
                             g["beta"][:, 0], dt_bias=g["dt_bias"])
    _close(y, ry[:, 0], "y")
    _close(state, rh, "state")


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("b,hk,h,K,V", [(80, 16, 32, 64, 64), (130, 10, 20, 128, 128), (300, 8, 8, 32, 96),
                                        (50, 25, 50, 72, 40), (40, 60, 60, 64, 256)])
def test_step_large_batch(cuda_ok, b, hk, h, K, V, io):
    """Enough rows and heads that CTAs stay for several of them: padding among
    the rows, slices, slots anywhere."""
    d = I.gdr_inputs(b, 1, hk, h, K, V, io=io, seed=b)
    g = _dev(d)
    qkv = torch.cat([g[x][:, 0].flatten(1) for x in ("q", "k", "v")], -1)
    q, k, v = qkv.split([hk * K, hk * K, h * V], -1)
    cache = 0.3 * torch.randn(b + 5, h, K, V, device="cuda")
    before = cache.clone()
    slots = torch.randperm(b + 5, generator=torch.Generator().manual_seed(b))[:b].to(torch.int32)
    slots[[1, 2, 7, b - 1]] = -1
    slots[b // 2] = b + 5
    live = [i for i in range(b) if 0 <= slots[i] < b + 5]
    y = torch.full((b, h, V), 7.0, dtype=v.dtype, device="cuda")
    _ops().gdr_scan_step(cache, q.unflatten(-1, (hk, K)), k.unflatten(-1, (hk, K)), v.unflatten(-1, (h, V)),
                         g["dt"][:, 0], g["A"], g["beta"][:, 0], dt_bias=g["dt_bias"], slots=slots.cuda(), y=y)
    at = slots[live].long()
    sub = {x: d[x][live] for x in ("q", "k", "v", "dt", "beta")}
    ry, rh, _ = O.gdr_scan(sub["q"], sub["k"], sub["v"], sub["dt"], d["A"], sub["beta"], d["dt_bias"],
                           before[at.cuda()], scale=K ** -0.5)
    _close(y[live], ry[:, 0], "y")
    _close(cache[at.cuda()], rh, "state")
    dead = [i for i in range(b) if i not in live]
    assert (y[dead] == 7).all()
    rest = [i for i in range(b + 5) if i not in at.tolist()]
    assert torch.equal(cache[rest], before[rest])


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_step_slots_padding_slices(cuda_ok, io):
    b, hk, h, K, V = 7, 2, 4, 64, 64
    d = I.gdr_inputs(b, 1, hk, h, K, V, io=io, seed=2)
    g = _dev(d)
    qkv = torch.cat([g[x][:, 0].flatten(1) for x in ("q", "k", "v")], -1)
    q, k, v = qkv.split([hk * K, hk * K, h * V], -1)
    ba = torch.cat([g["beta"][:, 0], g["dt"][:, 0]], -1)
    beta, dt = ba.split([h, h], -1)
    cache = 0.3 * torch.randn(9, h, K, V, device="cuda")
    before = cache.clone()
    slots = torch.tensor([8, 0, -1, 3, 5, 9, -7], dtype=torch.int32, device="cuda")
    live = [0, 1, 3, 4]
    y = torch.full((b, h, V), 7.0, dtype=v.dtype, device="cuda")
    _ops().gdr_scan_step(cache, q.unflatten(-1, (hk, K)), k.unflatten(-1, (hk, K)), v.unflatten(-1, (h, V)), dt,
                         g["A"], beta, dt_bias=g["dt_bias"], slots=slots, y=y)
    at = slots[live].long()
    sub = {x: d[x][live] for x in ("q", "k", "v", "dt", "beta")}
    ry, rh, _ = O.gdr_scan(sub["q"], sub["k"], sub["v"], sub["dt"], d["A"], sub["beta"], d["dt_bias"], before[at],
                           scale=K ** -0.5)
    _close(y[live], ry[:, 0], "y")
    _close(cache[at], rh, "state")
    assert (y[[2, 5, 6]] == 7).all()
    rest = [i for i in range(9) if i not in at.tolist()]
    assert torch.equal(cache[rest], before[rest])


def test_steps_continue_a_scan(cuda_ok):
    """A prompt, then decode steps on its state, is the longer prompt."""
    d = I.gdr_inputs(2, 75, 1, 2, 128, 128, seed=21)
    ry, rh, _ = _ref(d)
    g = _dev(d)
    part = {x: (g[x][:, :70] if x in ("q", "k", "v", "dt", "beta") else g[x]) for x in g}
    y, h = _scan(part)
    _close(y, ry[:, :70], "y")
    for t in range(70, 75):
        yt = _ops().gdr_scan_step(h, g["q"][:, t], g["k"][:, t], g["v"][:, t], g["dt"][:, t], g["A"],
                                  g["beta"][:, t], dt_bias=g["dt_bias"])
        _close(yt, ry[:, t], "y %d" % t)
    _close(h, rh, "state")


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("tokens,h,W", [(1, 1, 1), (3, 2, 7), (5, 3, 64), (130, 5, 128), (9, 1, 256), (4, 2, 77),
                                        (2, 3, 96), (3, 1, 1024), (2, 2, 8192), (1000, 3, 40)])
def test_head_norm(cuda_ok, tokens, h, W, io):
    dtype = {"f32": torch.float32, "bf16": torch.bfloat16}[io]
    g = torch.Generator().manual_seed(W)
    x = torch.randn(tokens, h, W, generator=g).to(dtype)
    wide = torch.randn(tokens, h * W + 8, generator=g).to(dtype)
    z = wide[:, :h * W].unflatten(-1, (h, W))
    w = 1 + 0.1 * torch.randn(W, generator=g)
    f = _ops().gdr_gated_rmsnorm_fwd
    # float32: the mean's sum and a few roundings, below 1e-5 of the value;
    # the hardware tanh of the bfloat16 gate is within a few 2^-11 of z
    _close(f(x.cuda(), wide.cuda()[:, :h * W].unflatten(-1, (h, W)), w.cuda()), O.head_rmsnorm(x, z, w), "gated")
    _close(f(x.cuda()), O.head_rmsnorm(x), "plain")
    _close(f(x.cuda(), None, w.cuda(), eps=0.5), O.head_rmsnorm(x, None, w, 0.5), "weight")
    xc = x.cuda()
    assert f(xc, z.cuda(), out=xc) is xc
    _close(xc, O.head_rmsnorm(x, z), "in place")


def test_head_norm_zero_row(cuda_ok):
    x = torch.zeros(2, 1, 64, device="cuda")
    assert (_ops().gdr_gated_rmsnorm_fwd(x) == 0).all()


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("W", [1, 2, 3, 4])
@pytest.mark.parametrize("C", [64, 12, 331])
def test_conv_packed(cuda_ok, C, W, io):
    dtype = {"f32": torch.float32, "bf16": torch.bfloat16}[io]
    lengths = [1, 40, 0, 2, 3, 31, 32, 33, 1, 64, 100]
    total, n = sum(lengths), len(lengths)
    g = torch.Generator().manual_seed(C + W)
    wide = torch.randn(total + 5, C + 8, generator=g).to(dtype)
    wide[total:] = float("nan")
    w, bias = torch.randn(C, W, generator=g), torch.randn(C, generator=g)
    cache = torch.randn(n + 3, C, W - 1, generator=g)
    slots = torch.randperm(n + 3, generator=g)[:n].to(torch.int32)
    cu = torch.tensor([0] + lengths).cumsum(0).to(torch.int32)
    u = torch.full((total + 5, C), 7.0, dtype=dtype).cuda()
    got = cache.cuda()
    x = wide[:, :C]
    _, state = _ops().ssm_conv1d_packed_fwd(wide.cuda()[:, :C], w.cuda(), bias.cuda(), got, cu_seqlens=cu.cuda(),
                                            slots=slots.cuda(), u=u)
    assert state is got
    ru, rs = O.conv1d_packed(x[:total], w, bias, cache[slots.long()], lengths)
    # float32: W + 3 roundings; bfloat16: its rounding and the hardware tanh
    _close(u[:total], ru, "u")
    assert (u[total:] == 7).all()
    assert torch.equal(got.cpu()[slots.long()].double(), torch.from_numpy(rs).reshape(n, C, W - 1))
    rest = [i for i in range(n + 3) if i not in slots.tolist()]
    assert torch.equal(got.cpu()[rest], cache[rest])
    # no state, no bias, no gate
    u2, none = _ops().ssm_conv1d_packed_fwd(x[:total].cuda(), w.cuda(), cu_seqlens=cu.cuda(), silu=False)
    assert none is None
    _close(u2, O.conv1d_packed(x[:total], w, None, None, lengths, act=False)[0], "plain")


def test_conv_packed_bad_bounds(cuda_ok):
    x = torch.randn(50, 64, device="cuda")
    w = torch.randn(64, 4, device="cuda")
    state = torch.randn(4, 64, 3, device="cuda")
    before = state.clone()
    u = torch.full((50, 64), 7.0, device="cuda")
    cu = torch.tensor([0, 20, 90, 90, 100], dtype=torch.int32, device="cuda")
    slots = torch.tensor([1, 0, 2, 3], dtype=torch.int32, device="cuda")
    _ops().ssm_conv1d_packed_fwd(x, w, None, state, cu_seqlens=cu, slots=slots, u=u)
    assert (u[20:] == 7).all() and (u[:20] != 7).all()
    assert torch.equal(state[[0, 2, 3]], before[[0, 2, 3]]) and torch.equal(state[1], x[17:20].T)


def test_conv_packed_equals_dense(cuda_ok):
    """Equal lengths through both convolutions, and the decode form."""
    ops = _ops()
    d = _dev(I.conv_inputs(3, 70, 64, io="bf16", seed=1, state=True))
    u, so = ops.ssm_conv1d_fwd(d["x"], d["w"], d["bias"], d["state"])
    cu = torch.arange(0, 211, 70, dtype=torch.int32, device="cuda")
    state = d["state"].clone()
    up, _ = ops.ssm_conv1d_packed_fwd(d["x"].reshape(210, 64), d["w"], d["bias"], state, cu_seqlens=cu)
    assert torch.equal(up.reshape(3, 70, 64), u) and torch.equal(state, so)
    x1 = d["x"][:, 0].contiguous()
    a, b = so.clone(), so.clone()
    u1, _ = ops.ssm_conv1d_fwd(x1[:, None], d["w"], d["bias"], a, in_place=True)
    u2, _ = ops.ssm_conv1d_packed_fwd(x1, d["w"], d["bias"], b,
                                      cu_seqlens=torch.arange(4, dtype=torch.int32, device="cuda"))
    assert torch.equal(u2, u1[:, 0]) and torch.equal(a, b)


def test_mixer_prompt_then_decode(cuda_ok):
    """The operators as a mixer uses them: packed prompts through the
    convolution, the scan and the norm, then decode steps in a padded batch,
    against the definitions over the whole sequences."""
    ops = _ops()
    hk, h, K, V, W = 1, 2, 64, 64, 4
    C = 2 * hk * K + h * V
    lengths, extra = [33, 70, 2], 2
    g = torch.Generator().manual_seed(31)
    bf = torch.bfloat16
    xs = [torch.randn(n + extra, C, generator=g).to(bf) for n in lengths]
    gates = [torch.randn(n + extra, 2 * h, generator=g).to(bf) for n in lengths]
    zs = [torch.randn(n + extra, h, V, generator=g).to(bf) for n in lengths]
    w, bias = torch.rand(C, W, generator=g) - 0.5, torch.rand(C, generator=g) - 0.5
    A, dt_bias = -1 - 4 * torch.rand(h, generator=g), torch.randn(h, generator=g) - 3
    weight = 1 + 0.1 * torch.randn(V, generator=g)
    slots = torch.tensor([4, 1, 2], dtype=torch.int32)
    conv_cache, cache = torch.zeros(5, C, W - 1).cuda(), torch.zeros(5, h, K, V).cuda()

    def split(u):
        q, k, v = u.split([hk * K, hk * K, h * V], -1)
        return q.unflatten(-1, (hk, K)), k.unflatten(-1, (hk, K)), v.unflatten(-1, (h, V))

    cat = [torch.cat([t[i][:n] for i, n in enumerate(lengths)]).cuda() for t in (xs, gates, zs)]
    cu = torch.tensor([0] + lengths).cumsum(0).to(torch.int32).cuda()
    u, _ = ops.ssm_conv1d_packed_fwd(cat[0], w.cuda(), bias.cuda(), conv_cache, cu_seqlens=cu, slots=slots.cuda())
    q, k, v = split(u[None])
    beta, dt = cat[1][None].split([h, h], -1)
    y, _ = ops.gdr_chunk_scan_fwd(q, k, v, dt, A.cuda(), beta, dt_bias=dt_bias.cuda(), h0=cache, cu_seqlens=cu,
                                  slots=slots.cuda(), h_last=cache)
    out = [ops.gdr_gated_rmsnorm_fwd(y[0], cat[2], weight.cuda()).split(lengths)]
    padded = torch.cat([slots, torch.tensor([-1], dtype=torch.int32)]).cuda()
    one = torch.arange(5, dtype=torch.int32, device="cuda")
    for t in range(extra):
        x, gt, z = (torch.cat([s[n + t][None] for s, n in zip(src, lengths)] + [src[0][:1] * 0]).cuda()
                    for src in (xs, gates, zs))
        u, _ = ops.ssm_conv1d_packed_fwd(x, w.cuda(), bias.cuda(), conv_cache, cu_seqlens=one, slots=padded,
                                         u=torch.zeros_like(x))
        q, k, v = split(u)
        beta, dt = gt.split([h, h], -1)
        y = ops.gdr_scan_step(cache, q, k, v, dt, A.cuda(), beta, dt_bias=dt_bias.cuda(), slots=padded,
                              y=torch.zeros(4, h, V, dtype=bf, device="cuda"))
        out.append(ops.gdr_gated_rmsnorm_fwd(y, z, weight.cuda())[:3, None].unbind(0))
    for i, n in enumerate(lengths):
        got = torch.cat([part[i] for part in out])
        u, _ = O.conv1d_packed(xs[i], w, bias, None, [n + extra])
        u = torch.from_numpy(u).to(bf)  # the tensors between the operators are bfloat16
        q, k, v = split(u[None])
        ry, rh, _ = O.gdr_scan(q, k, v, gates[i][None, :, h:], A, gates[i][None, :, :h], dt_bias, None,
                               scale=K ** -0.5)
        rn = O.head_rmsnorm(torch.from_numpy(ry[0]).to(bf), zs[i], weight)
        # an input of the scan may round to the other side of a step (2^-7 of
        # it), and so may y: four roundings in a row, each 2^-8, of the largest
        assert np.abs(_np(got) - rn).max() <= 4 * 2.0 ** -8 * np.abs(rn).max(), i
        assert np.abs(_np(cache[slots[i]]) - rh[0]).max() <= 4 * 2.0 ** -8 * np.abs(rh).max(), i


def test_host_tensors(cuda_ok):
    """Host tensors go through the same calls, states updated where they lie."""
    ops = _ops()
    d = I.gdr_inputs(2, 20, 1, 2, 64, 64, io="f32", seed=41, h0=True)
    ry, rh, states = _ref(d)
    y, h = _scan(d)
    assert not y.is_cuda and not h.is_cuda
    _close(y, ry, "y")
    _close(h, rh, "h_last")
    cache = d["h0"].clone()
    _, out = _scan({**d, "h0": cache}, h_last=cache)
    assert out is cache
    _close(cache, rh, "cache")
    state = d["h0"].clone()
    y1 = ops.gdr_scan_step(state, d["q"][:, 0], d["k"][:, 0], d["v"][:, 0], d["dt"][:, 0], d["A"], d["beta"][:, 0],
                           dt_bias=d["dt_bias"])
    _close(y1, ry[:, 0], "step y")
    _close(state, states[:, 0], "step state")
    x = torch.randn(4, 2, 32)
    _close(ops.gdr_gated_rmsnorm_fwd(x, x), O.head_rmsnorm(x, x), "norm")
    xc, w, st = torch.randn(6, 8), torch.randn(8, 4), torch.randn(2, 8, 3)
    ru, rs = O.conv1d_packed(xc, w, None, st, [2, 4])
    u, so = ops.ssm_conv1d_packed_fwd(xc, w, None, st, cu_seqlens=torch.tensor([0, 2, 6], dtype=torch.int32))
    _close(u, ru, "u")
    assert so is st and np.array_equal(_np(st), rs)


@pytest.mark.parametrize("io,L", [("f32", 200), ("bf16", 20), ("bf16", 200)])
def test_scan_not_a_number_stays_in_its_head(cuda_ok, io, L):
    """A value, key or gate that is not a number is seen in its own sequence and
    heads from its chunk on, and nowhere else."""
    for name in ("v", "k", "dt", "beta"):
        d = I.gdr_inputs(2, L, 2, 4, 64, 64, io=io, seed=3, h0=True)
        ry, rh, _ = _ref(d)
        at = L - 5
        d[name][0, at, 1] = float("nan")
        heads = [2, 3] if name == "k" else [1]
        y, h = _scan(_dev(d))
        assert torch.isnan(h[0, heads]).any() and torch.isnan(y[0, at:, heads]).any(), name
        ok = [i for i in range(4) if i not in heads]
        _close(y[:, :, ok], ry[:, :, ok], "y " + name)
        _close(h[:, ok], rh[:, ok], "state " + name)
        _close(y[1], ry[1], "the other sequence " + name)
        _close(y[0, :at // 64 * 64], ry[0, :at // 64 * 64], "chunks before " + name)


@pytest.mark.parametrize("io,L", [("f32", 100), ("bf16", 10), ("bf16", 100)])
def test_zero_rows_without_eps(cuda_ok, io, L):
    """Rows of zeros have nothing to normalise by, also with l2_eps 0."""
    d = I.gdr_inputs(1, L, 1, 1, 64, 64, io=io, seed=6, h0=True)
    d["k"][:, 3:6] = 0
    d["q"][:, 2:8] = 0
    y, h = _scan(_dev(d), l2_eps=0.0)
    ry, rh, _ = _ref(d, l2_eps=1e-30)
    _close(y, ry, "y")
    _close(h, rh, "h_last")


def test_scan_packed_many(cuda_ok):
    """More sequences than are put in order or looked through."""
    g = torch.Generator().manual_seed(1)
    for n in (300, 1100):
        lengths = (torch.rand(n, generator=g) * 4).int().tolist()
        lengths[5], lengths[n - 3] = 150, 70
        d = I.gdr_inputs(1, sum(lengths), 1, 1, 64, 64, io="bf16", seed=n)
        cu = torch.tensor([0] + lengths).cumsum(0).to(torch.int32).cuda()
        y, h = _scan(_dev(d), cu_seqlens=cu)
        for i in (0, 5, 6, n // 2, n - 3, n - 1):
            s = slice(sum(lengths[:i]), sum(lengths[:i + 1]))
            if s.stop == s.start:
                assert (h[i] == 0).all()
                continue
            part = {x: d[x][:, s] for x in ("q", "k", "v", "dt", "beta")}
            ry, rh, _ = O.gdr_scan(part["q"], part["k"], part["v"], part["dt"], d["A"], part["beta"], d["dt_bias"],
                                   None, scale=8 ** -1.0)
            _close(y[:, s], ry, "y %d" % i)
            _close(h[i][None], rh, "state %d" % i)


def _apart(bounds, rows):
    """The live sequences of `bounds`, or None where two of them overlap."""
    live = [(i, b, e) for i, (b, e) in enumerate(zip(bounds, bounds[1:])) if 0 <= b < e <= rows]
    spans = sorted((b, e) for _, b, e in live)
    return None if any(x[1] > y[0] for x, y in zip(spans, spans[1:])) else live


def _sets_going_back(rows, count, seed):
    g = np.random.default_rng(seed)
    sets = [[128, 192, 0, 128], [128, 256, 0, 128], [640, 700, 64, 320, 10, 30], [320, 400, 192, 300, 0, 150]]
    while len(sets) < count:
        bounds = [int(x) for x in g.integers(0, rows + 1, g.integers(3, 9))]
        if any(b > e for b, e in zip(bounds, bounds[1:])) and _apart(bounds, rows):
            sets.append(bounds)
    return sets


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_scan_bounds_going_back(cuda_ok, io):
    """Sequences apart from one another whose bounds lie in any order: each is
    what it is by itself; the pairs out of order hand their states on, and rows
    of no sequence stay."""
    rows, H, K = 1024, 1, 8
    d = I.gdr_inputs(1, rows, 1, H, K, K, io=io, seed=2)
    g = _dev(d)
    sets = _sets_going_back(rows, 240, seed=6)
    h0 = 0.3 * torch.randn(len(sets), 8, H, K, K, generator=torch.Generator().manual_seed(3))
    got, want = [], []
    for bounds, h in zip(sets, h0):
        n = len(bounds) - 1
        y = torch.full((1, rows, H, K), 7.0, dtype=g["v"].dtype, device="cuda")
        g["h0"] = h[:n].cuda()
        cu = torch.tensor(bounds, dtype=torch.int32, device="cuda")
        got.append((y, _scan(g, cu_seqlens=cu, y=y)[1]))
        want += [(b, e, h[i]) for i, b, e in _apart(bounds, rows)]
    at = 0
    ref = []
    for part in (want[i:i + 100] for i in range(0, len(want), 100)):
        longest = max(e - b for b, e, _ in part)
        row = torch.stack([torch.arange(longest).clamp(max=e - b - 1) + b for b, e, _ in part])
        x = {k: d[k][0][row] for k in ("q", "k", "v", "dt", "beta")}
        ry, _, states = O.gdr_scan(x["q"], x["k"], x["v"], x["dt"], d["A"], x["beta"], d["dt_bias"],
                                   torch.stack([h for _, _, h in part]), scale=K ** -0.5)
        ref += [(ry[i, :e - b], states[i, e - b - 1]) for i, (b, e, _) in enumerate(part)]
    for bounds, h, (y, out) in zip(sets, h0, got):
        live = _apart(bounds, rows)
        rest = torch.ones(rows, dtype=torch.bool)
        for i, b, e in live:
            _close(y[0, b:e], ref[at][0], "y %s %d" % (bounds, i))
            _close(out[i], ref[at][1], "state %s %d" % (bounds, i))
            rest[b:e] = False
            at += 1
        none = [i for i in range(len(bounds) - 1) if i not in [j for j, _, _ in live]]
        assert torch.equal(out[none].cpu(), h[none]), bounds
        assert (y[0, rest.cuda()] == 7).all(), bounds
    assert at == len(ref)


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_scan_mixed_strengths(cuda_ok, io):
    """Write strengths below zero in one chunk and none in the next, whose key
    lies along a state that is the same in all its rows: what is read of it is
    sqrt(K) times its values."""
    d = I.gdr_inputs(1, 200, 1, 1, 128, 64, io=io, seed=15, h0=True)
    d["h0"][:] = 1
    d["dt"] = None
    d["beta"][:] = 0.5
    d["beta"][:, :64] = 2.0 ** -30
    d["beta"][:, 5] = -2.0 ** -30
    d["k"][:, 64] = 1
    d["v"] = d["v"] * 2.0 ** -20
    y, h = _scan(_dev(d), flags=16)
    ry, rh, _ = _ref(d, flags=16)
    _close(y, ry, "y")
    _close(h, rh, "h_last")


@pytest.mark.parametrize("flags", [17, 25])
@pytest.mark.parametrize("L", [3000, 8192])
def test_scan_few_long_strengths(cuda_ok, L, flags):
    """Long sequences whose write strengths are numbers as they come: tokens of
    strength 4 under a key of their own, which the state does not hold and
    whose values are zero, so that nothing grows but what is not there."""
    K, V = 64, 64
    d = I.gdr_inputs(1, L, 1, 1, K, V, io="bf16", seed=L, h0=True)
    d["A"] = d["A"] * 1e-4
    if not flags & 8:
        d["beta"] = d["beta"].float().sigmoid().to(d["beta"].dtype)
        d["k"][..., 0] = 0
        d["h0"][:, :, 0] = 0
        at = slice(7, None, 64)
        d["k"][:, at] = 0
        d["k"][:, at, :, 0] = 1
        d["v"][:, at] = 0
        d["beta"][:, at] = 4
    y, h = _scan(_dev(d), flags=flags)
    ry, rh, _ = _ref(d, flags=flags)
    _close(y, ry, "y")
    _close(h, rh, "h_last")


def test_scan_workspace_of_the_caller(cuda_ok):
    """One that is large enough is used, a small one replaced; what is not the
    memory it counts, or lies elsewhere, is refused before anything runs."""
    ops = _ops()
    d = _dev(I.gdr_inputs(1, 200, 1, 2, 64, 64, seed=16))
    y0, h0 = _scan(d)
    space = torch.zeros(1 << 20, dtype=torch.uint8, device="cuda")
    y, h = _scan(d, workspace=space)
    assert torch.equal(y, y0) and torch.equal(h, h0) and (space != 0).any()
    y, h = _scan(d, workspace=space[:64])
    assert torch.equal(y, y0) and torch.equal(h, h0)
    for bad in (space[:1].expand(1 << 20), space[::2], space.cpu()):
        with pytest.raises(ValueError):
            _scan(d, workspace=bad)
    with pytest.raises(ops.L.SsmError):  # off 16 bytes
        _scan(d, workspace=space[8:])
    host = {k: None if x is None else x.cpu() for k, x in d.items()}
    y, h = _scan(host, workspace=space)
    assert torch.equal(y, y0.cpu()) and torch.equal(h, h0.cpu())
    with pytest.raises(ValueError):
        _scan(host, workspace=space.cpu())


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("rows,C", [(1024, 64), (1024, 5), (60, 64), (60, 5)])
def test_conv_packed_bounds_going_back(cuda_ok, rows, C, io):
    """As test_scan_bounds_going_back, in both forms (few sequences, and many
    for their rows)."""
    dtype = {"f32": torch.float32, "bf16": torch.bfloat16}[io]
    g = torch.Generator().manual_seed(rows + C)
    x = torch.randn(rows, C, generator=g).to(dtype)
    w, bias = torch.randn(C, 4, generator=g), torch.randn(C, generator=g)
    sets = [s for s in _sets_going_back(rows, 60, seed=C) if max(s) <= rows]
    assert any(rows < 16 * (len(s) - 1) for s in sets) == (rows == 60)
    for bounds in sets:
        n = len(bounds) - 1
        state = torch.randn(n, C, 3, generator=g)
        u = torch.full((rows, C), 7.0, dtype=dtype).cuda()
        got = state.cuda()
        _ops().ssm_conv1d_packed_fwd(x.cuda(), w.cuda(), bias.cuda(), got, u=u,
                                     cu_seqlens=torch.tensor(bounds, dtype=torch.int32, device="cuda"))
        rest = torch.ones(rows, dtype=torch.bool)
        want = state.double().numpy()
        for i, b, e in _apart(bounds, rows):
            ru, rs = O.conv1d_packed(x[b:e], w, bias, state[i:i + 1], [e - b])
            _close(u[b:e], ru, "u %s %d" % (bounds, i))
            want[i] = rs[0]
            rest[b:e] = False
        assert np.array_equal(_np(got), want), bounds
        assert (u[rest.cuda()] == 7).all(), bounds


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("W", [1, 2, 3, 4])
@pytest.mark.parametrize("C", [64, 12, 331])
def test_conv_packed_short_runs(cuda_ok, C, W, io):
    """The form for sequences that are short on average: some of several of its
    runs among them, histories and states from x, from the old state and both."""
    dtype = {"f32": torch.float32, "bf16": torch.bfloat16}[io]
    lengths = [1, 7, 8, 9, 17, 33, 0, 1, 2, 3, 1, 1, 2, 16, 64, 3] + [1, 2, 3, 0] * 8
    total, n = sum(lengths), len(lengths)
    assert total + 5 < 16 * n
    g = torch.Generator().manual_seed(C + W)
    wide = torch.randn(total + 5, C + 8, generator=g).to(dtype)
    wide[total:] = float("nan")
    w, bias = torch.randn(C, W, generator=g), torch.randn(C, generator=g)
    cache = torch.randn(n + 3, C, W - 1, generator=g)
    slots = torch.randperm(n + 3, generator=g)[:n].to(torch.int32)
    skip = [4, 20]
    index = slots.clone()
    index[skip[0]], index[skip[1]] = -1, n + 3
    cu = torch.tensor([0] + lengths).cumsum(0).to(torch.int32)
    u = torch.full((total + 5, C), 7.0, dtype=dtype).cuda()
    got = cache.cuda()
    _ops().ssm_conv1d_packed_fwd(wide.cuda()[:, :C], w.cuda(), bias.cuda(), got, cu_seqlens=cu.cuda(),
                                 slots=index.cuda(), u=u)
    ru, rs = O.conv1d_packed(wide[:total, :C], w, bias, cache[slots.long()], lengths)
    live = torch.cat([torch.full((m,), i not in skip) for i, m in enumerate(lengths)])
    # float32: W + 3 roundings; bfloat16: its rounding and the hardware tanh
    _close(u[:total][live.cuda()], ru[live.numpy()], "u")
    assert (u[:total][~live.cuda()] == 7).all() and (u[total:] == 7).all()
    on = [i for i in range(n) if i not in skip]
    assert torch.equal(got.cpu()[slots.long()[on]].double(), torch.from_numpy(rs).reshape(n, C, W - 1)[on])
    rest = [i for i in range(n + 3) if i not in slots[on].tolist()]
    assert torch.equal(got.cpu()[rest], cache[rest])


@pytest.mark.parametrize("long", [1, 40000])
@pytest.mark.parametrize("C", [64, 13])
def test_conv_packed_many(cuda_ok, C, long):
    """More sequences than are looked through, in both forms."""
    g = torch.Generator().manual_seed(C)
    n = 1500
    lengths = (torch.rand(n, generator=g) * 4).int().tolist()
    lengths[5], lengths[n - 3] = 150, long
    total = sum(lengths)
    assert (total < 16 * n) == (long == 1)
    x, w, state = torch.randn(total, C, generator=g), torch.randn(C, 4, generator=g), torch.randn(n, C, 3, generator=g)
    cu = torch.tensor([0] + lengths).cumsum(0).to(torch.int32).cuda()
    got = state.cuda()
    u, _ = _ops().ssm_conv1d_packed_fwd(x.cuda(), w.cuda(), None, got, cu_seqlens=cu)
    ru, rs = O.conv1d_packed(x, w, None, state, lengths)
    _close(u, ru, "u")
    assert torch.equal(got.cpu().double(), torch.from_numpy(rs))


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("raw", [False, True])
def test_scan_small_strengths(cuda_ok, raw, io):
    """Write strengths of some 4e-5 throughout: the state, small beside the
    values, keeps its digits."""
    d = I.gdr_inputs(1, 200, 1, 2, 128, 64, io=io, seed=17)
    d["beta"] = d["beta"] - 10
    if raw:
        d["beta"] = d["beta"].float().sigmoid().to(d["beta"].dtype)
    flags = 17 if raw else 25
    y, h = _scan(_dev(d), flags=flags)
    ry, rh, _ = _ref(d, flags=flags)
    _close(y, ry, "y")
    _close(h, rh, "h_last")


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("L,K", [(1829, 128), (6000, 64)])
def test_scan_few_long_untouched(cuda_ok, L, K, io):
    """Without decay, under one key: what the entering state holds beside it is
    handed from segment to segment as it is."""
    d = I.gdr_inputs(2, L, 1, 1, K, 64, io=io, seed=18, h0=True)
    d["dt"] = None
    d["k"][:] = d["k"][:, :1]
    y, h = _scan(_dev(d))
    ry, rh, _ = _ref(d)
    _close(y, ry, "y")
    _close(h, rh, "h_last")
