"""Host-only checks of the gated delta rule's operators: what the C ABI and
the binding refuse, before anything is launched, and the float64 definitions
against closed forms.  No GPU; fake device addresses are never dereferenced."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import gdr as O
from selective_state_space_28_b200 import _lib as L
from selective_state_space_28_b200 import build as B
from selective_state_space_28_b200 import inputs as I
from selective_state_space_28_b200 import ops

OK, NULL, SHAPE, DTYPE, ALIGN, UNSUP, WS = 0, 1, 2, 3, 4, 5, 6
P = 0x7f0000001000
FAR = 0x7f1000000000


@pytest.fixture(scope="module")
def lib():
    B.build()
    return L.lib()


def _scan(**kw):
    d = dict(batch=1, seqlen=64, heads=4, key_heads=2, key_dim=128, value_dim=128, sequences=1,
             state_rows=1, io=1, flags=25, scale=0.1, l2_eps=1e-6, q=P, k=P, v=P, dt=P, beta=P, A=P,
             y=FAR)
    d.update(kw)
    return L.GdrScanArgs(**d)


@pytest.mark.parametrize("kw,status", [
    (dict(q=None), NULL), (dict(k=None), NULL), (dict(v=None), NULL), (dict(beta=None), NULL),
    (dict(A=None), NULL), (dict(y=None), NULL), (dict(io=2), DTYPE), (dict(heads=0), SHAPE),
    (dict(key_heads=3), SHAPE), (dict(key_dim=0), SHAPE), (dict(value_dim=0), SHAPE),
    (dict(batch=-1), SHAPE), (dict(seqlen=-1), SHAPE), (dict(sequences=2), SHAPE),
    (dict(batch=2, sequences=1, cu_seqlens=P), SHAPE), (dict(flags=2), UNSUP), (dict(flags=32), UNSUP),
    (dict(key_dim=257), UNSUP), (dict(scale=float("nan")), SHAPE), (dict(scale=float("inf")), SHAPE),
    (dict(l2_eps=-1.0), SHAPE), (dict(l2_eps=float("nan")), SHAPE), (dict(q=P + 8), ALIGN),
    (dict(dt=P + 1), ALIGN), (dict(cu_seqlens=P + 2), ALIGN), (dict(h0=P + 4), ALIGN),
    (dict(q_row=255), SHAPE), (dict(v_row=511), SHAPE), (dict(dt_row=3), SHAPE),
    (dict(y=P + 64 * 256), SHAPE),  # y inside k's rows
    (dict(h0=FAR + (1 << 30), h_last=FAR + (1 << 30) + 64), SHAPE),
    (dict(h0=FAR + (1 << 30), state_rows=0), SHAPE),
    (dict(seqlen=1 << 31), UNSUP), (dict(state_rows=1 << 31), UNSUP),
])
def test_scan_rejects(lib, kw, status):
    assert lib.gdr_chunk_scan_fwd(ctypes.byref(_scan(**kw)), None) == status


def test_scan_null_and_empty(lib):
    n = ctypes.c_size_t(7)
    assert lib.gdr_chunk_scan_fwd(None, None) == NULL
    assert lib.gdr_chunk_scan_workspace(None, ctypes.byref(n)) == NULL
    assert lib.gdr_chunk_scan_workspace(ctypes.byref(_scan()), None) == NULL
    # the query looks at no pointer
    a = _scan(q=None, k=None, v=None, dt=None, beta=None, A=None, y=None)
    assert lib.gdr_chunk_scan_workspace(ctypes.byref(a), ctypes.byref(n)) == OK
    none = _scan(batch=0, sequences=0, q=None, k=None, v=None, dt=None, beta=None, A=None, y=None)
    assert lib.gdr_chunk_scan_fwd(ctypes.byref(none), None) == OK


def _step(**kw):
    d = dict(batch=4, heads=4, key_heads=2, key_dim=128, value_dim=128, state_rows=4, io=1, flags=25,
             scale=0.1, l2_eps=1e-6, q=P, k=P, v=P, dt=P, beta=P, A=P, state_io=FAR, y=FAR + (1 << 30))
    d.update(kw)
    return L.GdrStepArgs(**d)


@pytest.mark.parametrize("kw,status", [
    (dict(state_io=None), NULL), (dict(y=None), NULL), (dict(q=None), NULL), (dict(io=9), DTYPE),
    (dict(key_heads=0), SHAPE), (dict(state_rows=3), SHAPE), (dict(flags=4), UNSUP),
    (dict(key_dim=300), UNSUP), (dict(v=P + 2), ALIGN), (dict(slots=P + 1), ALIGN),
    (dict(y=P), SHAPE), (dict(k_row=100), SHAPE),
])
def test_step_rejects(lib, kw, status):
    assert lib.gdr_scan_step(ctypes.byref(_step(**kw)), None) == status


def test_step_empty_batch(lib):
    a = _step(batch=0, q=None, k=None, v=None, dt=None, beta=None, A=None, state_io=None, y=None)
    assert lib.gdr_scan_step(ctypes.byref(a), None) == OK


def _norm(**kw):
    d = dict(tokens=8, heads=2, width=128, io=1, flags=0, eps=1e-5, x=P, z=P + (1 << 20), out=FAR)
    d.update(kw)
    return L.GdrNormArgs(**d)


@pytest.mark.parametrize("kw,status", [
    (dict(width=0), SHAPE), (dict(heads=0), SHAPE), (dict(tokens=-1), SHAPE), (dict(eps=-1.0), SHAPE),
    (dict(eps=float("nan")), SHAPE), (dict(io=3), DTYPE), (dict(flags=1), UNSUP), (dict(width=8193), UNSUP),
    (dict(x=None), NULL), (dict(out=None), NULL), (dict(z=P + 4), ALIGN), (dict(out=P + 256), SHAPE),
    (dict(out=P + (1 << 20)), SHAPE), (dict(z_row=255), SHAPE),
])
def test_norm_rejects(lib, kw, status):
    assert lib.gdr_gated_rmsnorm_fwd(ctypes.byref(_norm(**kw)), None) == status


def _conv(**kw):
    d = dict(tokens=32, channels=64, width=4, sequences=2, state_rows=2, io=1, flags=1, x=P, w=P + (1 << 20),
             state_io=P + (1 << 21), cu_seqlens=P + (1 << 22), u=FAR)
    d.update(kw)
    return L.ConvPackedArgs(**d)


@pytest.mark.parametrize("kw,status", [
    (dict(width=0), SHAPE), (dict(width=5), UNSUP), (dict(channels=0), SHAPE), (dict(tokens=-1), SHAPE),
    (dict(io=4), DTYPE), (dict(flags=2), UNSUP), (dict(w=None), NULL), (dict(x=None), NULL), (dict(u=None), NULL),
    (dict(cu_seqlens=None), NULL), (dict(x=P + 2), ALIGN), (dict(u=P + 64), SHAPE), (dict(state_rows=1), SHAPE),
    (dict(x_row=63), SHAPE), (dict(state_io=FAR + 16), SHAPE), (dict(slots=P + 3), ALIGN),
])
def test_conv_rejects(lib, kw, status):
    assert lib.ssm_conv1d_packed_fwd(ctypes.byref(_conv(**kw)), None) == status


def test_conv_nothing_to_do(lib):
    assert lib.ssm_conv1d_packed_fwd(ctypes.byref(_conv(sequences=0, cu_seqlens=None)), None) == OK
    assert lib.ssm_conv1d_packed_fwd(ctypes.byref(_conv(tokens=0, x=None, u=None)), None) == OK


def test_binding_refuses():
    d = I.gdr_inputs(1, 8, 1, 2, 16, 16, io="f32", h0=True)

    def scan(**kw):
        e = {**d, **{k: kw.pop(k) for k in list(kw) if k in d}}
        return ops.gdr_chunk_scan_fwd(e["q"], e["k"], e["v"], e["dt"], e["A"], e["beta"], dt_bias=e["dt_bias"],
                                      h0=e["h0"], **kw)

    with pytest.raises(TypeError):
        scan(k=d["k"].bfloat16())
    with pytest.raises(TypeError):
        scan(A=d["A"].double())
    with pytest.raises(ValueError):
        scan(beta=d["beta"][:, :4])
    with pytest.raises(ValueError):
        scan(h0=d["h0"][:, :1])
    with pytest.raises(TypeError):
        scan(cu_seqlens=torch.tensor([0, 8]))
    with pytest.raises(ValueError):  # a cache to write to is needed
        scan(cu_seqlens=torch.tensor([0, 8], dtype=torch.int32), slots=torch.zeros(1, dtype=torch.int32))
    with pytest.raises(ValueError):
        ops.gdr_scan_step(d["h0"].mT, d["q"][:, 0], d["k"][:, 0], d["v"][:, 0], d["dt"][:, 0], d["A"],
                          d["beta"][:, 0])
    with pytest.raises(ValueError):
        ops.gdr_gated_rmsnorm_fwd(d["v"], d["v"][:, :4])
    with pytest.raises(ValueError):
        ops.ssm_conv1d_packed_fwd(d["v"][0, :, 0], torch.zeros(8, 4), cu_seqlens=torch.zeros(2, dtype=torch.int32))


@pytest.mark.parametrize("make,inner,row", [
    (lambda t: t, 2, 0),
    (lambda t: torch.cat([t, t], -1).flatten(2)[..., :24].unflatten(-1, (3, 8)), 2, 48),
    (lambda t: t.transpose(1, 2).contiguous().transpose(1, 2), 2, None),  # heads outermost: copied
    (lambda t: t[:, :1], 2, 120), (lambda t: t[:1, 1:], 2, 0), (lambda t: t[:, 1:], 2, None),
])
def test_row_views(make, inner, row):
    t = make(torch.arange(2 * 5 * 3 * 8, dtype=torch.float32).reshape(2, 5, 3, 8))
    out, got = ops._rows(t, inner, 4)
    assert torch.equal(out, t)
    if row is None:
        assert got == 0 and out.is_contiguous()
    else:
        assert got == row and out.data_ptr() == t.data_ptr()


def test_oracle_without_delta_is_the_ssd():
    """Keys that never meet (one axis each): the delta term is zero and the
    rule is a decayed sum of outer products."""
    rng = np.random.default_rng(0)
    K, V = 6, 3
    k = np.eye(K)[None, :, None]
    q, v = rng.normal(size=(1, K, 1, K)), rng.normal(size=(1, K, 1, V))
    dt, beta, A = rng.normal(size=(1, K, 1)), rng.normal(size=(1, K, 1)), np.array([-0.7])
    y, S, _ = O.gdr_scan(q, k, v, dt, A, beta, scale=1.0, flags=1)
    a = np.exp(np.logaddexp(0, dt[0, :, 0]) * A[0])
    for t in range(K):
        ref = sum(np.prod(a[s + 1:t + 1]) * beta[0, s, 0] * q[0, t, 0, s] * v[0, s, 0] for s in range(t + 1))
        assert np.allclose(y[0, t, 0], ref)


def test_oracle_full_strength_recalls():
    """Written at full strength under a unit key, a value is read back whole
    and replaces what the key held."""
    rng = np.random.default_rng(1)
    k = rng.normal(size=(1, 4, 1, 5))
    k[:, 3] = k[:, 1]
    v = rng.normal(size=(1, 4, 1, 2))
    y, S, _ = O.gdr_scan(k, k, v, None, None, np.ones((1, 4, 1)), scale=1.0, flags=16, l2_eps=0.0)
    assert np.allclose(y, v)


def test_scan_wants_its_workspace(lib):
    """The tensor-core shapes need one, the others do not; too small is refused."""
    n = ctypes.c_size_t(1)
    for kw, need in ((dict(seqlen=640), True), (dict(seqlen=640, io=0), False), (dict(seqlen=640, key_dim=132), False),
                     (dict(seqlen=640, q_row=260, key_dim=64), False), (dict(seqlen=640, value_dim=100), False),
                     (dict(seqlen=16), False)):
        a = _scan(**kw)
        assert lib.gdr_chunk_scan_workspace(ctypes.byref(a), ctypes.byref(n)) == OK
        assert (n.value > 0) == need, kw
    a = _scan(seqlen=640)
    lib.gdr_chunk_scan_workspace(ctypes.byref(a), ctypes.byref(n))
    assert lib.gdr_chunk_scan_fwd(ctypes.byref(a), None) == WS
    a.workspace, a.workspace_bytes = P, n.value - 1
    assert lib.gdr_chunk_scan_fwd(ctypes.byref(a), None) == WS


@pytest.mark.parametrize("pack,cls,name", [
    (L.GDR_SCAN, L.GdrScanArgs, "gdr_scan_args"), (L.GDR_STEP, L.GdrStepArgs, "gdr_step_args"),
    (L.GDR_NORM, L.GdrNormArgs, "gdr_norm_args"), (L.CONV_PACKED, L.ConvPackedArgs, "ssm_conv_packed_args")])
def test_packed_arguments_are_the_structures(pack, cls, name):
    """Every field lands where the C structure has it."""
    fields = cls._fields_
    for at in range(len(fields)):
        values = [0.0 if t is ctypes.c_float else 0 for _, t in fields]
        values[at] = 1.5 if fields[at][1] is ctypes.c_float else 77
        got = cls.from_buffer_copy(pack(*values))
        for (field, t), v in zip(fields, values):
            assert (getattr(got, field) or 0) == v, (name, field)


@pytest.mark.parametrize("kw", [dict(), dict(q=None, k=None, v=None, beta=None, y=None), dict(cu_seqlens=P)])
def test_scan_steps_need_their_rates(lib, kw):
    """Also where there is no token, and only the states are handed on."""
    assert lib.gdr_chunk_scan_fwd(ctypes.byref(_scan(seqlen=0, A=None, **kw)), None) == NULL


HERE = FAR + (1 << 32)  # a place of its own


@pytest.mark.parametrize("kw", [
    dict(y=HERE, h0=HERE + 1024), dict(y=HERE, h_last=HERE + 1024), dict(y=HERE, h0=HERE, h_last=HERE),
    dict(y=HERE, A=HERE), dict(y=HERE, dt_bias=HERE + 16), dict(y=HERE, slots=HERE + 64),
    dict(y=HERE, cu_seqlens=HERE + 4), dict(h_last=HERE, q=HERE + 16), dict(h_last=HERE, beta=HERE + 64),
    dict(h_last=HERE, h0=HERE, v=HERE), dict(h_last=HERE, slots=HERE + 8), dict(h_last=HERE + 16, A=HERE + 16),
])
def test_scan_rejects_overlap(lib, kw):
    """Outputs on inputs or on one another; that h_last is h0 is no overlap."""
    assert lib.gdr_chunk_scan_fwd(ctypes.byref(_scan(**kw)), None) == SHAPE


@pytest.mark.parametrize("name", ["q", "v", "dt", "A", "y", "h0", "h_last", "cu_seqlens", "slots"])
def test_scan_rejects_overlap_with_its_workspace(lib, name):
    a = _scan(seqlen=640)
    n = ctypes.c_size_t()
    setattr(a, name, HERE + 4096)
    assert lib.gdr_chunk_scan_workspace(ctypes.byref(a), ctypes.byref(n)) == OK
    a.workspace, a.workspace_bytes = HERE, n.value
    assert lib.gdr_chunk_scan_fwd(ctypes.byref(a), None) == SHAPE


@pytest.mark.parametrize("kw", [
    dict(y=FAR + 16), dict(state_io=P), dict(state_io=P, y=HERE), dict(q=FAR + 4096), dict(beta=FAR + 64),
    dict(A=FAR + 64), dict(dt_bias=FAR + (1 << 30) + 64), dict(slots=FAR + 4), dict(slots=FAR + (1 << 30)),
])
def test_step_rejects_overlap(lib, kw):
    assert lib.gdr_scan_step(ctypes.byref(_step(**kw)), None) == SHAPE


@pytest.mark.parametrize("kw", [
    dict(u=P + (1 << 20)), dict(u=P + (1 << 22)), dict(bias=FAR + 64), dict(slots=FAR + 4), dict(w=P + (1 << 21)),
    dict(bias=P + (1 << 21)), dict(slots=P + (1 << 21) + 4), dict(cu_seqlens=P + (1 << 21)),
])
def test_conv_rejects_overlap(lib, kw):
    assert lib.ssm_conv1d_packed_fwd(ctypes.byref(_conv(**kw)), None) == SHAPE


def test_binding_refuses_a_workspace_on_the_host():
    d = I.gdr_inputs(1, 80, 1, 1, 64, 64, io="bf16")
    for space in (torch.empty(1 << 20, dtype=torch.uint8), torch.empty(1, dtype=torch.uint8)):
        with pytest.raises(ValueError, match="workspace"):
            ops.gdr_chunk_scan_fwd(d["q"], d["k"], d["v"], d["dt"], d["A"], d["beta"], workspace=space)
