"""Linear attention's and beam search's entry points without a GPU: every refusal
comes from the host checks, before any HIP call, and empty problems succeed."""

import ctypes
import math
import os

import pytest

from distilled_modal_ssm_amd import binding as hb

FAKE = 0x10000  # never dereferenced: every call below ends in the host checks
BAD, NO, WS = hb.HM_ERR_INVALID_ARG, hb.HM_ERR_UNSUPPORTED, hb.HM_ERR_WORKSPACE


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not os.path.exists(hb.LIB_PATH):
        from distilled_modal_ssm_amd import build
        build.build()
    return hb.load()


def _refused(status, call, *args, **kw):
    with pytest.raises(hb.HMError) as e:
        call(*args, **kw)
    assert e.value.status == status, (kw, e.value)


def _desc(**kw):
    base = dict(batch=2, heads=8, key_dim=64, value_dim=48, act_dtype=hb.HM_BF16, scale=0.125)
    later = {k: kw.pop(k) for k in ("abi_version", "reserved") if k in kw}
    d = hb.make_linattn_desc(**{**base, **kw})
    for k, v in later.items():
        setattr(d, k, v)
    return d


DESCS = [
    (dict(abi_version=9), BAD), (dict(reserved=1), BAD), (dict(act_dtype=5), NO), (dict(batch=-1), BAD),
    (dict(heads=0), BAD), (dict(q_heads=3), BAD), (dict(k_heads=16), BAD), (dict(v_heads=0), BAD),
    (dict(key_dim=0), BAD), (dict(key_dim=257), NO), (dict(value_dim=300), NO), (dict(value_dim=-1), BAD),
    (dict(scale=math.inf), BAD), (dict(scale=math.nan), BAD), (dict(batch=1 << 40), BAD),
]


def _prefill(desc, L=100, **kw):
    a = dict(lengths=None, q=FAKE, ld_q=512, k=FAKE, ld_k=512, v=FAKE, ld_v=384, log_decay=FAKE, ld_decay=8, y=FAKE,
             ld_y=384, state_in=None, state_out=FAKE, workspace=None, ws_bytes=0, stream=0)
    hb.hyena_linattn_prefill(desc, L, **{**a, **kw})


def _token(desc, **kw):
    a = dict(q=FAKE, ld_q=512, k=FAKE, ld_k=512, v=FAKE, ld_v=384, log_decay=FAKE, ld_decay=0, y=FAKE, ld_y=384,
             state_in=FAKE, src_rows=None, state_out=FAKE, stream=0)
    hb.hyena_linattn_decode_step(desc, **{**a, **kw})


@pytest.mark.parametrize("kw,status", DESCS)
def test_linattn_descriptor(kw, status):
    d = _desc(**kw)
    _refused(status, hb.hyena_linattn_prefill_workspace, d, 10)
    _refused(status, _prefill, d)
    _refused(status, _token, d)


ROWS = [
    (dict(q=None), BAD), (dict(k=None), BAD), (dict(v=None), BAD), (dict(y=None), BAD), (dict(state_out=None), BAD),
    (dict(q=FAKE + 1), NO), (dict(y=FAKE + 1), NO), (dict(state_out=FAKE + 2), NO), (dict(log_decay=FAKE + 2), NO),
    (dict(ld_q=511), BAD), (dict(ld_k=0), BAD), (dict(ld_v=-384), BAD), (dict(ld_y=383), BAD), (dict(ld_decay=7), BAD),
    (dict(ld_decay=-1), BAD), (dict(ld_q=1 << 50), BAD), (dict(state_in=FAKE + 1), NO),
]


@pytest.mark.parametrize("kw,status", ROWS)
def test_linattn_arguments(kw, status):
    _refused(status, _prefill, _desc(), **kw)
    _refused(status, _token, _desc(), **kw)


def test_linattn_own_arguments():
    _refused(BAD, _prefill, _desc(), L=-1)
    _refused(NO, _prefill, _desc(), L=1 << 40, ld_decay=0)
    _refused(NO, _prefill, _desc(), lengths=FAKE + 2)
    _refused(NO, _prefill, _desc(), ld_k=1 << 22)
    _refused(BAD, hb.hyena_linattn_prefill_workspace, _desc(), -1)
    _refused(BAD, _token, _desc(), state_in=None)
    _refused(BAD, _token, _desc(), src_rows=FAKE)  # in place
    _refused(NO, _token, _desc(), src_rows=FAKE + 1, state_out=2 * FAKE)
    st = hb.load().hyena_linattn_prefill_workspace(ctypes.byref(_desc()), 10, None)
    assert st == BAD


def test_linattn_workspace():
    """A long prompt of few heads is cut into segments, whose states need memory; a missing or small one is refused."""
    d = _desc(batch=1, heads=2, key_dim=128, value_dim=128)
    n = hb.hyena_linattn_prefill_workspace(d, 60000)
    assert n >= 0 and hb.hyena_linattn_prefill_workspace(_desc(batch=0), 60000) == 0
    assert hb.hyena_linattn_prefill_workspace(d, 1) == 0
    if n:
        _refused(WS, _prefill, d, L=60000, workspace=None)
        _refused(WS, _prefill, d, L=60000, workspace=FAKE, ws_bytes=n - 1)
        _refused(NO, _prefill, d, L=60000, workspace=FAKE + 16, ws_bytes=n)


def test_empty_problems_need_no_gpu():
    _prefill(_desc(batch=0), q=None, k=None, v=None, y=None, state_out=None)
    _token(_desc(batch=0), q=None, k=None, v=None, y=None, state_in=None, state_out=None)
    hb.hyena_beam_select(0, 4, 100, 4, hb.HM_F32, None, 100, None, None, -1, None, None, None, None, None, 0, stream=0)
    hb.hyena_beam_reorder(0, 4, None, [], [], stream=0)
    hb.hyena_beam_reorder(3, 4, None, [], [], stream=0)


SIZES = [(-1, 4, 100, 4, BAD), (1, 0, 100, 4, BAD), (1, 65, 100, 4, BAD), (1, 4, 0, 4, BAD), (1, 4, 100, 0, BAD),
         (1, 4, 100, 65, BAD), (1, 1, 3, 4, BAD), (1, 64, 1 << 26, 4, NO), (1 << 30, 4, 100, 4, NO),
         (1 << 22, 4, 1 << 24, 4, NO)]


@pytest.mark.parametrize("G,K,V,n,status", SIZES)
def test_beam_sizes(G, K, V, n, status):
    _refused(status, hb.hyena_beam_select_workspace, G, K, V, n)
    _refused(status, hb.hyena_beam_select, G, K, V, n, hb.HM_F32, FAKE, V, FAKE, None, -1, FAKE, FAKE, FAKE, FAKE, FAKE,
             1 << 40, stream=0)


def _select(**kw):
    a = dict(groups=2, beams=4, vocab=1000, select=4, dtype=hb.HM_F32, logits=FAKE, ld=1000, scores=FAKE, finished=None,
             end_token=-1, out_scores=FAKE, out_tokens=FAKE, out_parents=FAKE, out_finished=FAKE, workspace=FAKE,
             ws_bytes=1 << 30, stream=0)
    hb.hyena_beam_select(**{**a, **kw})


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=3), NO), (dict(ld=999), BAD), (dict(end_token=1000), BAD), (dict(end_token=-2), BAD),
    (dict(finished=FAKE), BAD), (dict(logits=None), BAD), (dict(scores=None), BAD), (dict(out_scores=None), BAD),
    (dict(out_tokens=None), BAD), (dict(out_parents=None), BAD), (dict(logits=FAKE + 2), NO),
    (dict(dtype=hb.HM_BF16, logits=FAKE + 1), NO), (dict(scores=FAKE + 1), NO), (dict(out_parents=FAKE + 2), NO),
    (dict(workspace=None), WS), (dict(ws_bytes=8), WS), (dict(workspace=FAKE + 8), NO), (dict(ld=1 << 50), BAD),
])
def test_beam_select_arguments(kw, status):
    _refused(status, _select, **kw)


@pytest.mark.parametrize("args,status", [
    ((2, 4, None, [FAKE], [16]), BAD), ((2, 4, FAKE + 1, [FAKE], [16]), NO), ((2, 4, FAKE, [None], [16]), BAD),
    ((2, 4, FAKE, [FAKE], [-1]), BAD), ((-2, 4, FAKE, [FAKE], [16]), BAD), ((2, 65, FAKE, [FAKE], [16]), BAD),
    ((65536, 4, FAKE, [FAKE], [16]), NO), ((1, 4, FAKE, [FAKE], [(1 << 36) + 1]), NO), ((2, 4, FAKE, [FAKE], [1 << 60]), BAD),
])
def test_beam_reorder_arguments(args, status):
    _refused(status, hb.hyena_beam_reorder, *args, stream=0)
    with pytest.raises(ValueError):
        hb.hyena_beam_reorder(2, 4, FAKE, [FAKE], [], stream=0)
    assert hb.load().hyena_beam_reorder(2, 4, FAKE, -1, None, None, None) == BAD
    assert hb.load().hyena_beam_reorder(2, 4, FAKE, 1, None, None, None) == BAD


def test_linattn_rows_of_a_launch():
    """Rows and heads that four value tiles of 512 threads each give a launch of 2^32 threads."""
    d, kw = _desc(batch=1 << 18, value_dim=256), dict(ld_v=2048, ld_y=2048)
    _refused(NO, _prefill, d, L=3, **kw)
    _refused(NO, _prefill, d, **kw)
    _refused(NO, _token, d, **kw)


@pytest.mark.parametrize("G,K,V", [(1 << 23, 1, 2), (1 << 21, 4, 2), (1 << 20, 4, 1 << 15), (1 << 17, 64, 2)])
def test_beam_sizes_of_a_launch(G, K, V):
    """Segments that a launch has no threads for are refused; half as many rows are not."""
    _refused(NO, hb.hyena_beam_select_workspace, G, K, V, 1)
    assert hb.hyena_beam_select_workspace(G // 2, K, V, 1) > 0


def test_beam_select_scores_in_place():
    """Only where every group's new scores take the place of its own."""
    _refused(BAD, _select, select=3)
    _refused(BAD, _select, select=8)
    _refused(WS, _select, workspace=None)


def test_beam_reorder_row_limit():
    _refused(NO, hb.hyena_beam_reorder, 1, 4, FAKE, [FAKE], [(1 << 33) + 1], stream=0)


@pytest.mark.parametrize("beams", [1, 2, 3, 64])
def test_beam_vocabulary_fits_32_bit_places(beams):
    """A row's last segment starts less than 8 places before the row and ends up to a whole segment
    past it; each place, and the 16 bytes from it on, has to have a 32-bit number."""
    most = ((1 << 31) - 1 - (1 << 14)) // beams
    for vocab in (most + 1, ((1 << 31) - 1) // beams - 1, ((1 << 31) - 1) // beams):
        _refused(NO, hb.hyena_beam_select_workspace, 1, beams, vocab, 1)
        _refused(NO, _select, groups=1, beams=beams, vocab=vocab, ld=vocab, select=1, ws_bytes=1 << 60)
    assert hb.hyena_beam_select_workspace(1, beams, most, 1) > 0
    for segment in (2048, 8192):
        segs = -(-(most + 7) // segment)
        assert segs * segment + 8 < 1 << 31


class _NoDevice:
    """Stands in for the binding's _On where there is no GPU: stream 1 is current."""

    def __init__(self, device, stream):
        pass

    def __enter__(self):
        return 1

    def __exit__(self, *exc):
        return None


def _scratch_users(monkeypatch):
    """Calls that use scratch memory on stream 1, in place of the library's: each returns the address it was given."""
    import torch
    from distilled_modal_ssm_amd import BeamSearch, LinearAttention
    seen = []
    monkeypatch.setattr(hb, "_On", _NoDevice)
    monkeypatch.setattr(hb, "hyena_linattn_prefill",
                        lambda desc, L, *a: seen.append((a[-3].data_ptr(), a[-3].numel())))
    attn = LinearAttention(1, 2, 16, 16, "f32", device="cpu")

    def prompt(L):
        x = torch.zeros(1, L, 32)
        attn.prefill(x, x, x, y=x, state_out=torch.zeros(1, 2, 16, 16))
        return seen[-1]

    beam = BeamSearch(2, 3, 50, device="cpu")
    beam._select = lambda *a: seen.append((a[-3], a[-2])) or hb.HM_OK

    def select(_):
        beam.select(torch.zeros(6, 50), torch.zeros(2, 3))
        return seen[-1]

    return {"prompt": (attn, prompt), "select": (beam, select)}


@pytest.mark.parametrize("user", ["prompt", "select"])
def test_captured_calls_have_scratch_of_their_own(monkeypatch, user):
    """A graph replays the addresses of its capture: they are not a buffer that the handle may replace by
    a longer one or give to another call, and no memory of a graph is kept for later calls."""
    import torch
    handle, call = _scratch_users(monkeypatch)[user]
    capturing = []
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: bool(capturing))
    capturing.append(1)
    at, n = call(5000)
    assert at and n > 0 and not handle._ws
    capturing.clear()
    eager = call(5000)[0]
    assert call(5000)[0] == eager and len(handle._ws) == 1
    capturing.append(1)
    assert call(5000)[0] != eager
    capturing.clear()
    assert call(5000)[0] == eager and len(handle._ws) == 1


def test_scratch_grows_for_longer_prompts(monkeypatch):
    import torch
    _, call = _scratch_users(monkeypatch)["prompt"]
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    sizes = [call(L)[1] for L in (2000, 60000, 2000)]
    assert sizes[0] < sizes[1] == sizes[2]


def test_captured_modal_prompts_have_scratch_of_their_own(monkeypatch):
    import numpy as np
    import torch
    op = hb.ModalHyena(np.zeros((2, 8, 2)), np.zeros((2, 8, 2)), np.zeros(2), 1, 64, "f32", device="cpu")
    capturing = []
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: bool(capturing))
    capturing.append(1)
    first, n = op.workspace(70000)
    assert n > 0 and first.numel() >= n and op._ws is None
    capturing.clear()
    eager = op.workspace(70000)[0]
    capturing.append(1)
    own = op.workspace(70000)[0]
    assert own.data_ptr() != eager.data_ptr()
    capturing.clear()
    assert op.workspace(70000)[0] is eager


@pytest.mark.parametrize("act", [hb.HM_F32, hb.HM_BF16])
@pytest.mark.parametrize("dims", [(32, 32), (64, 128), (128, 128), (256, 256)])
def test_long_prompts_of_few_heads_run_in_segments(act, dims):
    """Their states need memory (a first state, and one a segment, at least two); a missing, small or
    misaligned one is refused."""
    d = _desc(batch=1, heads=2, key_dim=dims[0], value_dim=dims[1], act_dtype=act)
    n = hb.hyena_linattn_prefill_workspace(d, 60000)
    assert n >= 2 * 2 * dims[0] * dims[1] * 4
    ld = dict(ld_q=512, ld_k=512, ld_v=512, ld_y=512, ld_decay=0)
    _refused(WS, _prefill, d, L=60000, workspace=None, ws_bytes=n, **ld)
    _refused(WS, _prefill, d, L=60000, workspace=FAKE, ws_bytes=n - 1, **ld)
    _refused(NO, _prefill, d, L=60000, workspace=FAKE + 16, ws_bytes=n, **ld)


def test_beam_select_finished_in_place():
    """As for the scores: only where every group's new bytes take the place of its own."""
    kw = dict(finished=FAKE, out_finished=FAKE, end_token=0, out_scores=2 * FAKE)
    _refused(BAD, _select, select=3, **kw)
    _refused(BAD, _select, select=8, **kw)
    _refused(WS, _select, select=4, workspace=None, **kw)
    _refused(WS, _select, select=8, workspace=None, **{**kw, "out_finished": 3 * FAKE})
