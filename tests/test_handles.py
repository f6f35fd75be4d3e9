"""Handles and their scratch memory without a GPU: the library's calls are stood in for, on tensors of the host.

A call queues several kernels that hand values on through its scratch memory, and ctypes
lets other threads run meanwhile.  Two threads on one stream (the default stream is the
same for all) must not queue theirs in between.
"""

import gc
import os
import subprocess
import sys
import threading
import time

import pytest

from distilled_modal_ssm_amd import binding as hb


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not os.path.exists(hb.LIB_PATH):
        from distilled_modal_ssm_amd import build
        build.build()
    return hb.load()


@pytest.mark.parametrize("first", ["torch", "library"])
def test_one_hip_runtime_in_a_process(first):
    """Whichever of torch and the library is loaded first: torch brings a runtime of its own."""
    pytest.importorskip("torch")
    if not os.path.exists("/proc/self/maps"):
        pytest.skip("no list of mapped files")
    both = ["import torch", "from distilled_modal_ssm_amd import binding; binding.load()"]
    code = both if first == "torch" else both[::-1]
    code += ["print(*sorted({l.split()[-1] for l in open('/proc/self/maps') if 'libamdhip64' in l}))"]
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    out = subprocess.run([sys.executable, "-c", "\n".join(code)], cwd=root, capture_output=True, text=True, timeout=300)
    assert out.returncode == 0, out.stderr
    assert len(out.stdout.split()) == 1, out.stdout


class _Library:
    """In place of the C entry points: a call queues two kernels on its scratch memory, a moment apart."""

    def __init__(self):
        self.queue = []  # (stream, workspace, thread)

    def __call__(self, *args):
        ws, _, stream = args[-3:]
        ws = getattr(ws, "data_ptr", lambda: ws)()
        for _ in range(2):
            self.queue.append((stream, ws, threading.get_ident()))
            time.sleep(0.001)
        return hb.HM_OK

    def check(self, calls):
        """What is queued on one stream's scratch memory comes in pairs of one thread's."""
        order = {}
        for stream, ws, thread in self.queue:
            order.setdefault((stream, ws), []).append(thread)
        assert sum(map(len, order.values())) == 2 * calls
        for threads in order.values():
            assert threads[::2] == threads[1::2], threads


def _users(torch, monkeypatch, library):
    """name -> a call that takes the stream and goes through a handle to ``library``."""
    from distilled_modal_ssm_amd import BeamSearch, DraftVerify, GatedRecurrence, Int8Dense, LinearAttention

    class On:
        def __init__(self, device, stream):
            self.stream = 0 if stream is None else stream

        def __enter__(self):
            return self.stream

        def __exit__(self, *exc):
            return None

    monkeypatch.setattr(hb, "_On", On)
    monkeypatch.setattr(hb, "_call", lambda call, device, stream, *args: call(*args, 0 if stream is None else stream))
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    monkeypatch.setattr(hb, "hyena_quantize_rows", lambda *a: None)
    monkeypatch.setattr(hb, "hyena_linattn_prefill", library)
    # (its arguments end in workspace, bytes, stream, chunk and algorithm)
    monkeypatch.setattr(hb, "hyena_modal_prefill", lambda *a: library(*a[:-2]))
    import numpy as np
    rec = GatedRecurrence(1, 16, "f32", device="cpu")
    rec._prompt = rec._grads = library
    verify = DraftVerify(2, 3, 5000, device="cpu")
    verify._verify = library
    dense = Int8Dense(torch.zeros(30, 100))
    dense._product = library
    attn = LinearAttention(1, 2, 16, 16, "f32", device="cpu")
    beam = BeamSearch(2, 3, 50, device="cpu")
    beam._select = library
    modal = hb.ModalHyena(np.zeros((2, 8, 2)), np.zeros((2, 8, 2)), np.zeros(2), 1, 64, "f32", device="cpu")
    x, wide, long = torch.zeros(1, 500, 16), torch.zeros(1, 5000, 32), torch.zeros(1, 70000, 64)
    chunks, state = torch.zeros(1, 8, 16), torch.zeros(1, 2, 16, 16)
    p, drafted, u = torch.zeros(2, 4, 5000), torch.zeros(2, 3, dtype=torch.int32), torch.zeros(2, 4)
    rows, logits, scores = torch.zeros(9, 100), torch.zeros(6, 50), torch.zeros(2, 3)
    return {
        "recurrence": lambda s: rec.prefill(x, x, x, stream=s),
        "gradients": lambda s: rec.backward(x, x, x, x, chunks, stream=s),
        "verify": lambda s: verify.verify(p, drafted, u, stream=s),
        "dense": lambda s: dense(rows, stream=s),
        "attention": lambda s: attn.prefill(wide, wide, wide, y=wide, state_out=state, stream=s),
        "beams": lambda s: beam.select(logits, scores, stream=s),
        "modal": lambda s: modal.prefill(long, long, long, y=long, stream=s),
    }


USERS = ["recurrence", "gradients", "verify", "dense", "attention", "beams", "modal"]


@pytest.mark.parametrize("user", USERS)
def test_threads_on_one_stream(monkeypatch, user):
    import torch
    library = _Library()
    call = _users(torch, monkeypatch, library)[user]
    calls, start = 8, threading.Barrier(2)

    def work():
        start.wait()
        for _ in range(calls):
            call(None)

    threads = [threading.Thread(target=work) for _ in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    library.check(2 * calls)


@pytest.mark.parametrize("user", USERS)
def test_streams_have_buffers_of_their_own(monkeypatch, user):
    """Their kernels run at the same time; a stream's next call finds its own again."""
    import torch
    library = _Library()
    call = _users(torch, monkeypatch, library)[user]
    for stream in (1, 2, None, 1, 2, None):
        call(stream)
    assert [s for s, _, _ in library.queue[::2]] == [1, 2, 0, 1, 2, 0]
    at = [ws for _, ws, _ in library.queue[::2]]
    assert at[:3] == at[3:] and len(set(at)) == 3


@pytest.mark.parametrize("user", USERS)
def test_a_refused_call_lets_the_next_one_in(monkeypatch, user):
    import torch

    def refuses(*args):
        raise hb.HMError(hb.HM_ERR_HIP, "call")

    library = _Library()
    answer = [refuses]
    call = _users(torch, monkeypatch, lambda *a: answer[0](*a))[user]
    with pytest.raises(hb.HMError):
        call(None)
    answer[0] = library
    done = threading.Thread(target=call, args=(None,), daemon=True)
    done.start()
    done.join(10)
    assert not done.is_alive()
    library.check(1)


def test_a_models_products_share_their_scratch(monkeypatch):
    """One buffer a device and stream, as long as the longest rows need, given back with the last handle."""
    import torch
    from distilled_modal_ssm_amd import Int8Dense
    library = _Library()
    _users(torch, monkeypatch, library)
    layers = [Int8Dense(torch.zeros(30, K)) for K in (100, 400, 200)]
    for layer in layers:
        layer._product = library
    for layer in (layers[1], layers[0], layers[2], layers[1]):
        layer(torch.zeros(50, layer.K), stream=1)
    assert len({ws for _, ws, _ in library.queue}) == 1
    layers[0](torch.zeros(9, 100), stream=2)
    assert len({ws for _, ws, _ in library.queue}) == 2
    pool = layers[0]._ws
    assert all(layer._ws is pool for layer in layers) and len(pool) == 2
    del pool, layer, layers
    gc.collect()
    again = Int8Dense(torch.zeros(30, 100))
    assert not again._ws


def test_fft_prompts_keep_their_scratch_on_their_stream(monkeypatch):
    """Its memory goes back to torch when the call returns, before its kernels have run: to the stream that runs them."""
    import numpy as np
    import torch
    current = []

    class On:
        def __init__(self, device, stream):
            self.stream = 0 if stream is None else stream

        def __enter__(self):
            current.append(self.stream)
            return self.stream

        def __exit__(self, *exc):
            current.pop()

    made, empty = [], torch.empty
    monkeypatch.setattr(hb, "_On", On)
    monkeypatch.setattr(torch, "empty", lambda *a, **kw: made.append(list(current)) or empty(*a, **kw))
    monkeypatch.setattr(hb, "hyena_fft_prefill", lambda *a: made.append(a[-1]))
    op = hb.ModalHyena(np.zeros((2, 8, 2)), np.zeros((2, 8, 2)), np.zeros(2), 1, 64, "f32", device="cpu")
    x = torch.zeros(1, 70000, 64)
    made.clear()
    op.fft_prefill(x, x, x, stream=7)
    assert made == [[7], [7], 7]


def test_a_module_in_torchs_place(monkeypatch):
    import types
    monkeypatch.setitem(sys.modules, "torch", types.ModuleType("torch"))
    hb._torch_runtime()
