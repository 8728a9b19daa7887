"""Refusals of the delta rule's and the state cache's entry points: on the host, before any launch."""
import ctypes
import math

import pytest

from mamba_ssd_scan_02_b200 import ssd

FAKE = 1 << 20  # never dereferenced: validation fails first


@pytest.fixture(scope="module")
def lib():
    return ssd.load()


def config(**kw):
    c = ssd.make_delta_config(dict(nheads=8, ngroups=2), 1, 100)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def args(**kw):
    a = ssd.DeltaArgs(q=FAKE, q_row_stride=256, k=FAKE, k_row_stride=256, v=FAKE, v_row_stride=512, dt=FAKE,
                      dt_row_stride=8, b=FAKE, b_row_stride=8, A=FAKE, dt_bias=FAKE, y=1 << 30, y_row_stride=512)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def test_struct_layout_matches_header(lib):
    assert ctypes.sizeof(ssd.DeltaConfig) == 16 * 4
    assert ctypes.sizeof(ssd.DeltaArgs) == 18 * 8
    assert ctypes.sizeof(ssd.DeltaDecodeArgs) == 17 * 8
    assert ctypes.sizeof(ssd.StateCacheArgs) == 9 * 8


@pytest.mark.parametrize("kw,status", [
    (dict(batch=0), 1), (dict(seqlen=-1), 1), (dict(nheads=6, ngroups=4), 1), (dict(ngroups=0), 1),
    (dict(headdim=32), 2), (dict(headdim=96), 2), (dict(dstate=64), 2), (dict(qk_eps=0.0), 1), (dict(qk_eps=math.nan), 1),
    (dict(qk_norm=2), 1), (dict(q_scale=math.inf), 1), (dict(beta_scale=math.nan), 1), (dict(dt_min=1.0, dt_max=0.5), 1),
    (dict(dt_min=math.nan), 1), (dict(io_dtype=2), 1), (dict(kernel=3), 1), (dict(kernel=2, io_dtype=0), 2),
    (dict(beta_sigmoid=5), 1), (dict(dt_softplus=-1), 1), (dict(batch=70000), 2), (dict(nheads=131072, ngroups=2), 2),
], ids=str)
def test_config_refused(lib, kw, status):
    c = config(**kw)
    assert lib.ssd_delta_prefill(ctypes.byref(c), ctypes.byref(args()), None) == status
    if "kernel" not in kw or kw["kernel"] == 3:
        assert lib.ssd_delta_workspace_size(ctypes.byref(c)) == 0
    if "seqlen" not in kw and "kernel" not in kw:
        d = ssd.DeltaDecodeArgs(state=FAKE, n_slots=1)
        assert lib.ssd_delta_decode_step(ctypes.byref(c), ctypes.byref(d), None) == status


@pytest.mark.parametrize("kw,status", [
    (dict(q=None), 1), (dict(k=None), 1), (dict(v=None), 1), (dict(dt=None), 1), (dict(b=None), 1), (dict(A=None), 1),
    (dict(dt_bias=None), 1), (dict(y=None), 1), (dict(q_row_stride=255), 1), (dict(v_row_stride=504), 1),
    (dict(y_row_stride=0), 1), (dict(dt_row_stride=7), 1), (dict(b_row_stride=-8), 1), (dict(q=FAKE + 8), 3),
    (dict(k_row_stride=260), 3), (dict(y=(1 << 30) + 2), 3), (dict(y_row_stride=516), 3), (dict(h0=FAKE + 4), 3),
    (dict(h_final=FAKE + 8), 3), (dict(dt=FAKE + 1), 3), (dict(A=FAKE + 2), 3),
    (dict(y=FAKE), 1),                                                     # the output over the inputs
    (dict(h0=1 << 40, h_final=(1 << 40) + 1024), 1),                       # states that overlap in part
], ids=str)
def test_arguments_refused(lib, kw, status):
    assert lib.ssd_delta_prefill(ctypes.byref(config()), ctypes.byref(args(**kw)), None) == status


def test_null_structs_refused(lib):
    assert lib.ssd_delta_prefill(None, None, None) == 1
    assert lib.ssd_delta_prefill(ctypes.byref(config()), None, None) == 1
    assert lib.ssd_delta_decode_step(None, None, None) == 1
    assert lib.ssd_delta_decode_step(ctypes.byref(config()), None, None) == 1
    assert lib.ssd_state_store(None, None) == 1 and lib.ssd_state_load(None, None) == 1
    assert lib.ssd_delta_prefill_varlen(ctypes.byref(config()), ctypes.byref(args()), None, 1, None) == 1


@pytest.mark.parametrize("cu", [[0, 60, 40, 100], [1, 100], [0, 99], [0, 101], [100]], ids=str)
def test_offsets_refused(lib, cu):
    arr = (ctypes.c_int * len(cu))(*cu)
    c = config()
    assert lib.ssd_delta_prefill_varlen(ctypes.byref(c), ctypes.byref(args()), arr, len(cu) - 1, None) == 1
    assert lib.ssd_delta_varlen_workspace_size(ctypes.byref(c), arr, len(cu) - 1) == 0
    ok = (ctypes.c_int * 3)(0, 40, 100)
    assert lib.ssd_delta_prefill_varlen(ctypes.byref(config(batch=2)), ctypes.byref(args()), ok, 2, None) == 1
    assert lib.ssd_delta_varlen_workspace_size(ctypes.byref(c), ok, 2) > 0
    assert lib.ssd_delta_prefill_varlen(ctypes.byref(c), ctypes.byref(args()), ok, 2, None) == 7  # no workspace


def test_columns_of_one_matrix_may_interleave(lib):
    """y beside v in the same rows passes the overlap check (and stops at the missing workspace)."""
    wide = dict(q=FAKE, q_row_stride=2048, k=FAKE + 512, k_row_stride=2048, v=FAKE + 1024, v_row_stride=2048,
                dt=FAKE + 3072, dt_row_stride=2048, b=FAKE + 3104, b_row_stride=2048, y_row_stride=2048)
    ok = (ctypes.c_int * 3)(0, 40, 100)
    c = config()
    call = lambda **kw: lib.ssd_delta_prefill_varlen(ctypes.byref(c), ctypes.byref(args(**wide, **kw)), ok, 2, None)
    assert call(y=FAKE + 2048) == 7
    assert call(y=FAKE + 2032) == 1  # its first columns are v's last
    assert call(y=FAKE + 2064) == 1  # its last columns are dt's first


def decode(**kw):
    a = ssd.DeltaDecodeArgs(q=FAKE, q_row_stride=256, k=FAKE, k_row_stride=256, v=FAKE, v_row_stride=512, dt=FAKE,
                            dt_row_stride=8, b=FAKE, b_row_stride=8, A=FAKE, dt_bias=FAKE, state=1 << 40, n_slots=4,
                            y=1 << 30, y_row_stride=512)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("kw,status", [
    (dict(state=None), 1), (dict(q=None), 1), (dict(n_slots=0), 1), (dict(n_slots=3), 1), (dict(state=(1 << 40) + 4), 3),
    (dict(slots=FAKE + 2), 3), (dict(v=FAKE + 4), 3), (dict(y_row_stride=511), 1), (dict(y=FAKE + 256), 1),
], ids=str)
def test_decode_refused(lib, kw, status):
    assert lib.ssd_delta_decode_step(ctypes.byref(config(batch=4)), ctypes.byref(decode(**kw)), None) == status


def cache(**kw):
    a = ssd.StateCacheArgs(format=0, state_elems=8192, count=4, n_states=4, n_cache=4, states=1 << 40, cache=1 << 30,
                           scales=1 << 28)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("kw,status", [
    (dict(format=2), 1), (dict(state_elems=0), 1), (dict(state_elems=8200), 1), (dict(count=-1), 1), (dict(states=None), 1),
    (dict(cache=None), 1), (dict(scales=None), 1), (dict(n_states=3), 1), (dict(n_cache=3), 1),
    (dict(n_states=0, state_slots=FAKE), 1), (dict(count=65536, n_states=65536, n_cache=65536), 2),
    (dict(states=(1 << 40) + 8), 3), (dict(cache=(1 << 30) + 4), 3), (dict(scales=(1 << 28) + 2), 3),
    (dict(state_slots=FAKE + 1), 3), (dict(cache_slots=FAKE + 2), 3),
    (dict(cache=(1 << 40) + 4 * 8192 * 4 - 16), 1), (dict(scales=(1 << 30) + 4), 1),
], ids=str)
def test_state_cache_refused(lib, kw, status):
    for call in (lib.ssd_state_store, lib.ssd_state_load):
        assert call(ctypes.byref(cache(**kw)), None) == status


def test_no_entries_is_no_work(lib):
    for call in (lib.ssd_state_store, lib.ssd_state_load):
        assert call(ctypes.byref(cache(count=0, states=None)), None) == 0


def test_binding_checks_shapes_and_types():
    import torch
    cfg = dict(nheads=2, ngroups=1)
    bf, f = torch.bfloat16, torch.float32
    z = lambda *s, dtype=bf: torch.zeros(*s, dtype=dtype)
    good = dict(q=z(1, 4, 128), k=z(1, 4, 128), v=z(1, 4, 128), dt=z(1, 4, 2), b=z(1, 4, 2), A=z(2, dtype=f), dt_bias=z(2, dtype=f))
    for name, bad in (("q", z(1, 4, 127)), ("k", z(1, 5, 128)), ("v", z(1, 4, 128, dtype=f)), ("dt", z(1, 4, 3)),
                      ("b", z(1, 4, 2, dtype=f)), ("A", z(3, dtype=f)), ("dt_bias", z(2)), ("q", z(4, 128)),
                      ("k", z(1, 4, 256)[..., ::2]), ("h0", z(1, 2, 64, 127, dtype=f))):
        with pytest.raises(ValueError):
            ssd.delta_prefill(cfg, **dict(good, **{name: bad}))
    with pytest.raises(ValueError, match="CUDA"):  # no fallback on the host
        ssd.delta_prefill(cfg, **good)
    with pytest.raises(ValueError):  # batch rows that are not evenly spaced
        two = {k: (v if v.dim() == 1 else torch.cat([v, v])) for k, v in good.items()}
        ssd.delta_prefill(cfg, **dict(two, q=z(2, 5, 128)[:, :4]))
    with pytest.raises(ValueError):
        ssd.delta_prefill_varlen(cfg, [0], *(z(4, 128) for _ in range(3)), z(4, 2), z(4, 2), good["A"], good["dt_bias"])
    with pytest.raises(ValueError):
        ssd.state_store(z(2, 4, 128, dtype=f), z(2, 4, 128), z(2, 4, 4, dtype=torch.uint8))
    with pytest.raises(ValueError):
        ssd.state_store(z(2, 4, 128, dtype=f), z(2, 4, 128, dtype=torch.int8), z(2, 4, 3, dtype=torch.uint8))
    with pytest.raises(ValueError):
        ssd.state_cache(1, (4, 100))
