"""The entry points of the gated recurrence, of 8-bit products and of draft verification without a
GPU: every refusal comes from the host checks, before any HIP call, and empty problems succeed."""

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
    assert e.value.status == status, (args, kw, e.value)


def _desc(**kw):
    version = kw.pop("abi_version", None)
    d = hb.make_recurrence_desc(**{**dict(batch=2, channels=96, act_dtype=hb.HM_BF16), **kw})
    if version is not None:
        d.abi_version = version
    return d


def _prompt(desc, L=100, **kw):
    a = dict(lengths=None, q=FAKE, ld_q=96, g=FAKE, ld_g=96, v=FAKE, ld_v=96, y=FAKE, ld_y=96, state_in=None,
             state_out=FAKE, chunk_states=None, workspace=FAKE, ws_bytes=1 << 40, stream=0)
    hb.hyena_recurrence_prefill(desc, L, **{**a, **kw})


def _backward(desc, L=100, **kw):
    a = dict(lengths=None, q=FAKE, ld_q=96, g=FAKE, ld_g=96, v=FAKE, ld_v=96, dy=FAKE, ld_dy=96, chunk_states=FAKE,
             dstate_out=None, dq=FAKE, ld_dq=96, dg=FAKE, ld_dg=96, dv=FAKE, ld_dv=96, dstate_in=None, workspace=FAKE,
             ws_bytes=1 << 40, stream=0)
    hb.hyena_recurrence_backward(desc, L, **{**a, **kw})


def _token(desc, **kw):
    a = dict(q=FAKE, ld_q=96, g=FAKE, ld_g=96, v=FAKE, ld_v=96, y=FAKE, ld_y=96, state_in=FAKE, src_rows=None,
             state_out=FAKE, stream=0)
    hb.hyena_recurrence_decode_step(desc, **{**a, **kw})


@pytest.mark.parametrize("kw,status", [
    (dict(abi_version=9), BAD), (dict(act_dtype=5), NO), (dict(batch=-1), BAD), (dict(channels=0), BAD),
    (dict(gate=2), BAD), (dict(gate=-1), BAD), (dict(input=3), BAD), (dict(input=-1), BAD), (dict(batch=1 << 45), BAD),
])
def test_recurrence_descriptor(kw, status):
    d = _desc(**kw)
    _refused(status, hb.hyena_recurrence_workspace, d, 10)
    for call in (_prompt, _backward, _token):
        _refused(status, call, d)


@pytest.mark.parametrize("kw,status", [
    (dict(g=None), BAD), (dict(v=None), BAD), (dict(q=FAKE + 1), NO), (dict(g=FAKE + 1), NO), (dict(v=FAKE + 1), NO),
    (dict(ld_q=95), BAD), (dict(ld_g=0), BAD), (dict(ld_v=-96), BAD), (dict(ld_v=1 << 46), BAD),
])
def test_recurrence_inputs(kw, status):
    for call in (_prompt, _backward, _token):
        _refused(status, call, _desc(), **kw)


def test_recurrence_own_arguments():
    for kw, status in ((dict(y=None), BAD), (dict(y=FAKE + 1), NO), (dict(ld_y=95), BAD), (dict(state_out=None), BAD),
                       (dict(state_out=FAKE + 2), NO), (dict(state_in=FAKE + 1), NO)):
        _refused(status, _prompt, _desc(), **kw)
        _refused(status, _token, _desc(), **kw)
    for call in (_prompt, _backward):
        _refused(BAD, call, _desc(), L=-1)
        _refused(NO, call, _desc(), L=1 << 30)
        _refused(NO, call, _desc(), lengths=FAKE + 2)
        _refused(NO, call, _desc(), chunk_states=FAKE + 2)
    for name in ("dq", "dg", "dv", "dy"):
        _refused(BAD, _backward, _desc(), **{name: None})
        _refused(NO, _backward, _desc(), **{name: FAKE + 1})
        _refused(BAD, _backward, _desc(), **{"ld_" + name: 95})
    _refused(BAD, _backward, _desc(), q=None)  # dq goes with q
    _refused(BAD, _backward, _desc(), chunk_states=None)
    _refused(NO, _backward, _desc(), dstate_out=FAKE + 1)
    _refused(NO, _backward, _desc(), dstate_in=FAKE + 1)
    _refused(BAD, _token, _desc(), state_in=None)
    _refused(BAD, _token, _desc(), src_rows=FAKE)  # in place
    _refused(NO, _token, _desc(), src_rows=FAKE + 1, state_out=2 * FAKE)
    _refused(BAD, hb.hyena_recurrence_workspace, _desc(), -1)
    assert hb.load().hyena_recurrence_workspace(ctypes.byref(_desc()), 10, None) == BAD


@pytest.mark.parametrize("ld", [1 << 22, 1 << 30])
def test_recurrence_strides(ld):
    """Rows too far apart for a wave's 32-bit offsets: of every tensor, where there are several."""
    d = _desc(batch=1)
    for name in ("q", "g", "v", "y"):
        _refused(NO, _prompt, d, L=2, **{"ld_" + name: ld})
    for name in ("q", "g", "v", "dy", "dq", "dg", "dv"):
        _refused(NO, _backward, d, L=2, **{"ld_" + name: ld})


@pytest.mark.parametrize("B,D,L", [(1 << 23, 1, 1), (1 << 20, 512, 1), (1 << 9, 64, 1 << 20), (1, 1 << 29, 1)])
def test_recurrence_sizes_of_a_launch(B, D, L):
    """Batch rows, channel tiles and chunks that a launch has no threads for are refused; half as many are not."""
    for call in (lambda d: hb.hyena_recurrence_workspace(d, L), lambda d: _prompt(d, L, ld_q=D, ld_g=D, ld_v=D, ld_y=D)):
        _refused(NO, call, _desc(batch=B, channels=D))
    assert hb.hyena_recurrence_workspace(_desc(batch=B // 2 or 1, channels=D if B > 1 else D // 2), L) >= 0


def test_recurrence_workspace():
    d = _desc()
    n = hb.hyena_recurrence_workspace(d, 100000)
    assert hb.hyena_recurrence_workspace(_desc(batch=0), 100000) == 0
    if n:
        for call in (_prompt, _backward):
            _refused(WS, call, d, L=100000, workspace=None)
            _refused(WS, call, d, L=100000, ws_bytes=n - 1)
            _refused(NO, call, d, L=100000, workspace=FAKE + 16)


def _quantize(**kw):
    a = dict(M=4, K=100, dtype=hb.HM_F32, x=FAKE, ldx=100, rms=0, eps=0.0, q=FAKE, scale=FAKE, stream=0)
    hb.hyena_quantize_rows(**{**a, **kw})


@pytest.mark.parametrize("kw,status", [
    (dict(M=-1), BAD), (dict(K=0), BAD), (dict(K=131073, ldx=1 << 18), NO), (dict(dtype=2), NO),
    (dict(rms=1, eps=-1.0), BAD), (dict(rms=1, eps=math.nan), BAD), (dict(rms=1, eps=math.inf), BAD), (dict(ldx=99), BAD),
    (dict(x=None), BAD), (dict(q=None), BAD), (dict(scale=None), BAD),
    (dict(x=FAKE + 2), NO), (dict(dtype=hb.HM_BF16, x=FAKE + 1), NO), (dict(q=FAKE + 8), NO), (dict(scale=FAKE + 2), NO),
    (dict(M=1 << 24), NO), (dict(M=1 << 23, ldx=1 << 24), BAD),
])
def test_quantize_arguments(kw, status):
    _refused(status, _quantize, **kw)


def test_int8_bytes():
    assert hb.hyena_int8_bytes(1, 1) == 1024 and hb.hyena_int8_bytes(33, 65) == 3 * 2 * 1024
    assert hb.hyena_int8_bytes(0, 5) == 0
    _refused(BAD, hb.hyena_int8_bytes, -1, 5)
    _refused(BAD, hb.hyena_int8_bytes, 5, 0)
    _refused(NO, hb.hyena_int8_bytes, 5, 131073)
    assert hb.load().hyena_int8_bytes(1, 1, None) == BAD


def _dense(**kw):
    a = dict(M=4, N=50, K=100, A=FAKE, a_scale=FAKE, W=FAKE, w_scale=FAKE, dtype=hb.HM_F32, C=FAKE, ldc=50, stream=0)
    hb.hyena_dense_int8(**{**a, **kw})


@pytest.mark.parametrize("kw,status", [
    (dict(M=-1), BAD), (dict(N=-1), BAD), (dict(K=0), BAD), (dict(K=131073), NO),
    (dict(dtype=7), NO), (dict(ldc=49), BAD), (dict(A=None), BAD), (dict(W=None), BAD), (dict(C=None), BAD),
    (dict(a_scale=None), BAD), (dict(w_scale=None), BAD), (dict(A=FAKE + 8), NO), (dict(W=FAKE + 4), NO),
    (dict(C=FAKE + 2), NO), (dict(a_scale=FAKE + 1), NO), (dict(w_scale=FAKE + 2), NO), (dict(M=(1 << 31) - 512), NO),
    (dict(N=(1 << 31) - 512, ldc=1 << 31), NO), (dict(M=1 << 19, N=1 << 19, ldc=1 << 19), NO),
    (dict(M=1 << 27, ldc=1 << 22), BAD),
])
def test_dense_int8_arguments(kw, status):
    _refused(status, _dense, **kw)


def _dense_rows(**kw):
    a = dict(M=4, N=50, K=100, x_dtype=hb.HM_F32, x=FAKE, ldx=100, rms=0, eps=0.0, W=FAKE, w_scale=FAKE, dtype=hb.HM_BF16,
             C=FAKE, ldc=50, workspace=FAKE, ws_bytes=1 << 30, stream=0)
    hb.hyena_dense_int8_rows(**{**a, **kw})


@pytest.mark.parametrize("kw,status", [
    (dict(M=-1), BAD), (dict(N=-1), BAD), (dict(K=0), BAD), (dict(K=131073, ldx=1 << 18), NO), (dict(dtype=7), NO),
    (dict(x_dtype=7), NO), (dict(ldc=49), BAD), (dict(ldx=99), BAD), (dict(x=None), BAD), (dict(W=None), BAD),
    (dict(C=None), BAD), (dict(w_scale=None), BAD), (dict(x=FAKE + 2), NO), (dict(W=FAKE + 4), NO), (dict(C=FAKE + 1), NO),
    (dict(w_scale=FAKE + 2), NO), (dict(rms=1, eps=-1.0), BAD), (dict(M=1 << 24), NO), (dict(workspace=None), WS),
    (dict(ws_bytes=2048), WS), (dict(workspace=FAKE + 64), NO), (dict(M=1 << 23, ldx=1 << 24), BAD),
])
def test_dense_int8_rows_arguments(kw, status):
    _refused(status, _dense_rows, **kw)


def test_dense_int8_rows_workspace():
    assert hb.hyena_dense_int8_rows_workspace(33, 65) == 3 * 2 * 1024 + 256
    assert hb.hyena_dense_int8_rows_workspace(0, 65) == 0
    _refused(BAD, hb.hyena_dense_int8_rows_workspace, 1, 0)
    assert hb.load().hyena_dense_int8_rows_workspace(1, 1, None) == BAD


def _verify(**kw):
    a = dict(batch=3, drafts=4, vocab=1000, dtype=hb.HM_F32, p=FAKE, ld_p=1000, q=FAKE, ld_q=1000, tokens=FAKE,
             lengths=None, u=FAKE, out_tokens=FAKE, out_accepted=FAKE, workspace=FAKE, ws_bytes=1 << 30, stream=0)
    hb.hyena_draft_verify(**{**a, **kw})


@pytest.mark.parametrize("kw,status", [
    (dict(batch=-1), BAD), (dict(drafts=-1), BAD), (dict(drafts=64), BAD), (dict(vocab=0), BAD),
    (dict(vocab=(1 << 31) - (1 << 14), ld_p=1 << 32, ld_q=1 << 32), NO), (dict(batch=1 << 23), NO), (dict(dtype=3), NO),
    (dict(p=None), BAD), (dict(tokens=None), BAD), (dict(u=None), BAD), (dict(out_tokens=None), BAD),
    (dict(out_accepted=None), BAD), (dict(ld_p=999), BAD), (dict(ld_q=999), BAD), (dict(p=FAKE + 2), NO),
    (dict(q=FAKE + 2), NO), (dict(dtype=hb.HM_BF16, q=FAKE + 1), NO), (dict(tokens=FAKE + 1), NO),
    (dict(lengths=FAKE + 2), NO), (dict(u=FAKE + 2), NO), (dict(out_tokens=FAKE + 1), NO), (dict(out_accepted=FAKE + 2), NO),
    (dict(workspace=None), WS), (dict(ws_bytes=8), WS), (dict(workspace=FAKE + 8), NO), (dict(ld_p=1 << 45), BAD),
])
def test_verify_arguments(kw, status):
    _refused(status, _verify, **kw)


def test_empty_problems_need_no_gpu():
    none = dict(q=None, g=None, v=None)
    _prompt(_desc(batch=0), **none, y=None, state_out=None)
    _backward(_desc(batch=0), **none, dy=None, dq=None, dg=None, dv=None, chunk_states=None)
    _token(_desc(batch=0), **none, y=None, state_in=None, state_out=None)
    _quantize(M=0, x=None, q=None, scale=None)
    _dense(M=0, A=None, a_scale=None, C=None)
    _dense(N=0, W=None, w_scale=None, C=None)
    _dense_rows(M=0, x=None, C=None, workspace=None, ws_bytes=0)
    _dense_rows(N=0, W=None, w_scale=None, C=None, workspace=None, ws_bytes=0)
    _verify(batch=0, p=None, q=None, tokens=None, u=None, out_tokens=None, out_accepted=None, workspace=None, ws_bytes=0)
    assert hb.hyena_draft_verify_workspace(0, 4, 1000) == 0
    assert hb.load().hyena_draft_verify_workspace(1, 4, 1000, None) == BAD


def _scratch_users(monkeypatch):
    """Calls that use scratch memory on stream 1, in place of the library's: each returns the address it was given."""
    import torch
    from distilled_modal_ssm_amd import DraftVerify, GatedRecurrence, Int8Dense
    seen = []
    monkeypatch.setattr(hb, "_call", lambda call, device, stream, *args: call(*args, 1))
    rec = GatedRecurrence(1, 16, "f32", device="cpu")
    rec._prompt = lambda *a: seen.append((a[-3], a[-2])) or hb.HM_OK

    def prompt(n):
        x = torch.zeros(1, n, 16)
        rec.prefill(x, x, x)
        return seen[-1]

    verify = DraftVerify(2, 3, 5000, device="cpu")
    verify._verify = lambda *a: seen.append((a[-3], a[-2])) or hb.HM_OK

    def check(_):
        verify.verify(torch.zeros(2, 4, 5000), torch.zeros(2, 3, dtype=torch.int32), torch.zeros(2, 4))
        return seen[-1]

    class OnHost:
        def __init__(self, *a):
            pass

        def __enter__(self):
            return 1

        def __exit__(self, *exc):
            return None

    monkeypatch.setattr(hb, "_On", OnHost)
    monkeypatch.setattr(hb, "hyena_quantize_rows", lambda *a: None)
    dense = Int8Dense(torch.zeros(30, 100))
    dense._product = lambda *a: seen.append((a[-3], a[-2])) or hb.HM_OK

    def product(n):
        dense(torch.zeros(n, 100))
        return seen[-1]

    return {"prompt": (rec, prompt), "verify": (verify, check), "dense": (dense, product)}


@pytest.mark.parametrize("user", ["prompt", "verify", "dense"])
def test_captured_calls_have_scratch_of_their_own(monkeypatch, user):
    """As for the other handles: a graph's addresses are not a buffer that a later call replaces or uses."""
    import torch
    handle, call = _scratch_users(monkeypatch)[user]
    capturing = [1]
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: bool(capturing))
    at, n = call(5000)
    assert at and n > 0 and not handle._ws
    capturing.clear()
    eager = call(5000)[0]
    assert call(5000)[0] == eager and len(handle._ws) == 1
    capturing.append(1)
    assert call(5000)[0] != eager
    capturing.clear()
    assert call(5000)[0] == eager and len(handle._ws) == 1


def test_recurrence_workspaces_of_short_and_long_prompts():
    """A workgroup's tokens (8, 64 or 128) need none; more are joined through words of 8 bytes a channel and place,
    the backward pass's of 64 tokens the most."""
    d = _desc(batch=3, channels=100)
    assert [hb.hyena_recurrence_workspace(d, L) for L in (0, 1, 8, 9, 64)] == [0] * 5
    assert hb.hyena_recurrence_workspace(d, 65) == 3 * 2 * 128 + 3 * 128 * (2 + 1 + 1) * 8
    places = -(-100000 // 64)
    groups = -(-places // 8)
    assert hb.hyena_recurrence_workspace(d, 100000) == 3 * 2 * 128 + 3 * 128 * (places + groups + -(-groups // 8)) * 8


def test_tensors_of_the_host_are_refused(monkeypatch):
    """Before any call of the library: its pointers are device pointers."""
    import torch
    from distilled_modal_ssm_amd import DraftVerify, GatedRecurrence, Int8Dense

    def never(*a):
        raise AssertionError("called")

    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    rec, verify = GatedRecurrence(1, 16, "f32", device="cpu"), DraftVerify(1, 1, 9, device="cpu")
    rec._prompt = rec._token = rec._grads = verify._verify = never
    monkeypatch.setattr(hb, "hyena_quantize_rows", never)
    x = torch.zeros(1, 3, 16)
    for call in (lambda: rec.prefill(x, x, x), lambda: rec.decode_step(x[:, 0], x[:, 0], x[:, 0], torch.zeros(1, 16)),
                 lambda: rec.backward(x, x, x, x, torch.zeros(1, 1, 16)), lambda: Int8Dense(torch.zeros(4, 4)),
                 lambda: verify.verify(torch.zeros(1, 2, 9), torch.zeros(1, 1, dtype=torch.int32), torch.zeros(1, 2))):
        with pytest.raises(ValueError):
            call()
