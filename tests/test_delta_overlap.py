"""Outputs and scratch that share memory with something else are refused on the host, before any launch."""
import ctypes

import pytest

from mamba_ssd_scan_02_b200 import ssd

# addresses that nothing dereferences: every call ends at a refusal or at a missing workspace
IN, H0, HF, Y, WS = 1 << 20, 1 << 40, 1 << 41, 1 << 30, 1 << 42
STATE = 2 * 8 * 64 * 128 * 4  # bytes of two sequences' states


@pytest.fixture(scope="module")
def lib():
    return ssd.load()


def prefill(lib, workspace=False, seqlen=100, **kw):
    """A packed call of two sequences; without a workspace it ends with SSD_ERR_WORKSPACE (7)."""
    c = ssd.make_delta_config(dict(nheads=8, ngroups=2), 1, seqlen)
    a = ssd.DeltaArgs(q=IN, q_row_stride=256, k=IN + (1 << 17), k_row_stride=256, v=IN + (1 << 18), v_row_stride=512,
                      dt=IN + (1 << 19), dt_row_stride=8, b=IN + (1 << 19) + 4096, b_row_stride=8, A=IN - 4096, dt_bias=IN - 2048,
                      h0=H0, y=Y, y_row_stride=512, h_final=HF)
    if workspace:
        a.workspace, a.workspace_bytes = WS, 1 << 30
    for k, v in kw.items():
        setattr(a, k, v)
    return lib.ssd_delta_prefill_varlen(ctypes.byref(c), ctypes.byref(a), (ctypes.c_int * 3)(0, seqlen // 2, seqlen), 2, None)


@pytest.mark.parametrize("kw", [
    dict(y=H0), dict(y=H0 + STATE - 16), dict(y=H0 - 100 * 1024 + 16), dict(y=HF), dict(y=HF + STATE - 16),
    dict(y=IN - 4096), dict(y=IN - 4096 - 100 * 1024 + 16), dict(y=IN - 2048 + 16),
    dict(h_final=IN), dict(h_final=IN + (1 << 17) + 64), dict(h_final=IN + (1 << 18) - STATE + 16), dict(h_final=IN + (1 << 19)),
    dict(h_final=IN - 4096 - STATE + 16), dict(h_final=H0 + 1024), dict(h_final=H0 - STATE + 16), dict(h_final=Y),
], ids=str)
def test_outputs_over_something_else(lib, kw):
    assert prefill(lib, **kw) == 1


@pytest.mark.parametrize("kw", [
    dict(), dict(h_final=H0), dict(h_final=None), dict(h0=None), dict(y=H0 + STATE), dict(y=H0 - 100 * 1024),
    dict(h_final=H0 + STATE), dict(h_final=H0 - STATE), dict(h_final=Y + 100 * 1024),
    dict(y=IN - 4096 - 100 * 1024),
], ids=str)
def test_neighbours_are_fine(lib, kw):
    assert prefill(lib, **kw) == 7


@pytest.mark.parametrize("kw", [
    dict(q=WS), dict(v=WS + 240), dict(dt=WS), dict(A=WS + 16), dict(h0=WS), dict(h0=WS - STATE + 16), dict(y=WS), dict(h_final=WS),
    dict(y=WS - 100 * 1024 + 16), dict(h_final=WS - STATE + 16, h0=None),
], ids=str)
def test_workspace_over_something_else(lib, kw):
    assert prefill(lib, workspace=True, **kw) == 1


def test_without_tokens_only_the_states_count(lib):
    # (what is not read may be anything: this one ends at the missing workspace)
    assert prefill(lib, seqlen=0, q=H0, A=HF, y=H0, h0=H0, h_final=H0) == 7
    assert prefill(lib, seqlen=0, h_final=H0 + 1024) == 1
    assert prefill(lib, seqlen=0, workspace=True, h_final=WS) == 1


def test_a_state_between_the_rows_of_a_wider_matrix(lib):
    """y as columns of a matrix in whose other columns, or behind whose rows, something else lies."""
    wide = dict(y=Y, y_row_stride=1 << 21)  # rows of 4 MB, 1 KB of them y
    assert prefill(lib, **wide, h_final=Y + 1024) == 7
    assert prefill(lib, **wide, h_final=Y + (1 << 22) - STATE) == 7
    assert prefill(lib, **wide, h_final=Y + 1024 - 16) == 1
    assert prefill(lib, **wide, h_final=Y + (1 << 22) - STATE + 16) == 1
    assert prefill(lib, **wide, h_final=Y + 99 * (1 << 22) + 1024) == 7
    assert prefill(lib, **wide, h_final=Y + 99 * (1 << 22) + 1008) == 1


def decode(lib, **kw):
    c = ssd.make_delta_config(dict(nheads=8, ngroups=2), 4, 1)
    a = ssd.DeltaDecodeArgs(q=IN, q_row_stride=256, k=IN + 8192, k_row_stride=256, v=IN + 16384, v_row_stride=512, dt=IN + 32768,
                            dt_row_stride=8, b=IN + 33000, b_row_stride=8, A=IN + 34048, dt_bias=IN + 35072, state=H0, n_slots=4,
                            slots=IN + 36096, y=Y, y_row_stride=512)
    for k, v in kw.items():
        setattr(a, k, v)
    return lib.ssd_delta_decode_step(ctypes.byref(c), ctypes.byref(a), None)


@pytest.mark.parametrize("kw", [
    dict(y=H0), dict(y=H0 + 2 * STATE - 16), dict(y=H0 - 4096 + 16), dict(y=IN + 34048 + 16), dict(y=IN + 36096), dict(y=IN + 35072 - 4096 + 1024),
    dict(state=IN), dict(state=IN - 2 * STATE + 16), dict(state=IN + 35072 - 2 * STATE + 16, A=IN + (1 << 23), q=IN + (1 << 24), k=IN + (1 << 25), v=IN + (1 << 26), dt=IN + (1 << 27), b=IN + (1 << 28)),
    dict(state=IN + 36096), dict(state=Y),
], ids=str)
def test_decode(lib, kw):
    assert decode(lib, **kw) == 1


def cache(lib, call, **kw):
    a = ssd.StateCacheArgs(format=0, state_elems=8192, count=4, n_states=4, n_cache=4, states=1 << 40, cache=1 << 30,
                           scales=1 << 28, state_slots=IN, cache_slots=IN + 64)
    for k, v in kw.items():
        setattr(a, k, v)
    return getattr(lib, call)(ctypes.byref(a), None)


def test_state_cache(lib):
    for slots in ("state_slots", "cache_slots"):
        assert cache(lib, "ssd_state_store", **{slots: (1 << 30) + 64}) == 1
        assert cache(lib, "ssd_state_store", **{slots: (1 << 28) + 64}) == 1
        assert cache(lib, "ssd_state_load", **{slots: (1 << 40) + 64}) == 1
    for call in ("ssd_state_store", "ssd_state_load"):
        # sizes whose bytes do not fit a 64-bit number
        assert cache(lib, call, state_elems=1 << 40, n_states=(1 << 31) - 1) == 2
        assert cache(lib, call, state_elems=1 << 40, n_cache=(1 << 31) - 1) == 2
