"""Handles used on two streams, and by two threads, at the same time: every call's results are those of the same
call alone, compared for equality (results do not depend on timing)."""

import threading

import pytest

from _gpu_common import log, require_gpu
from distilled_modal_ssm_amd import DraftVerify, GatedRecurrence, Int8Dense
from distilled_modal_ssm_amd import binding as hb

pytestmark = pytest.mark.gpu


def _users(torch):
    """name -> (a call of one handle on inputs and a stream, a function that makes inputs): all of several launches
    that hand values on through scratch memory."""
    g = torch.Generator(device="cuda").manual_seed(5)
    randn = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    rec = GatedRecurrence(3, 300, "bf16")
    dense = Int8Dense(randn(700, 900))
    verify = DraftVerify(5, 4, 70000)

    def train(x, stream):
        chunks = rec_chunks.pop()
        y = rec.prefill(*x[:3], chunk_states=chunks, stream=stream)
        return (*y, *rec.backward(*x, chunks, stream=stream))

    rec_chunks = [rec.new_chunk_states(3000) for _ in range(200)]
    probs = lambda *s: torch.softmax(3 * randn(*s, 70000), -1)  # noqa: E731
    from distilled_modal_ssm_amd import ModalHyena
    circle = 0.95 * torch.exp(1j * torch.linspace(0, 3, 16)).view(2, 8)
    poles, residues = (torch.view_as_real(t.to(torch.complex64)).contiguous() for t in (circle, circle / 8))
    modal = ModalHyena(poles, residues, torch.ones(2), 1, 128, "f32")
    return {
        "modal": (lambda x, stream: modal.prefill(*x, stream=stream), lambda: [randn(1, 20000, 128) for _ in range(3)]),
        "fft": (lambda x, stream: (modal.fft_prefill(*x, stream=stream),), lambda: [randn(1, 20000, 128) for _ in range(3)]),
        "train": (train, lambda: [randn(3, 3000, 300).bfloat16() for _ in range(4)]),
        "dense": (lambda x, stream: (dense(x[0], rms_eps=1e-6, stream=stream),), lambda: [randn(400, 900)]),
        "verify": (lambda x, stream: verify.verify(*x[:3], q=x[3], stream=stream),
                   lambda: [probs(5, 5), torch.randint(0, 70000, (5, 4), generator=g, device="cuda", dtype=torch.int32),
                            torch.rand(5, 5, generator=g, device="cuda"), probs(5, 4)]),
    }


@pytest.mark.parametrize("user", ["train", "dense", "verify", "modal", "fft"])
def test_two_streams_at_once(user):
    torch = require_gpu()
    log(f"two streams {user}")
    call, new = _users(torch)[user]
    inputs = [new(), new()]
    want = [call(x, None) for x in inputs]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(6):
        for k in (0, 1):
            got[k].append(call(inputs[k], streams[k]))
    torch.cuda.synchronize()
    for k in (0, 1):
        for out in got[k]:
            assert all(torch.equal(a, b) for a, b in zip(out, want[k])), k
    assert not torch.equal(want[0][0], want[1][0])


@pytest.mark.parametrize("user", ["train", "dense", "verify", "modal", "fft"])
def test_two_threads_on_one_stream(user):
    torch = require_gpu()
    log(f"two threads {user}")
    call, new = _users(torch)[user]
    inputs = [new(), new()]
    want = [call(x, None) for x in inputs]
    torch.cuda.synchronize()
    got, start = [[], []], threading.Barrier(2)

    def work(k):
        start.wait()
        for _ in range(30):
            got[k].append(call(inputs[k], None))

    threads = [threading.Thread(target=work, args=(k,)) for k in (0, 1)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    for k in (0, 1):
        assert len(got[k]) == 30
        for out in got[k]:
            assert all(torch.equal(a, b) for a, b in zip(out, want[k])), k


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("L", [5, 64, 65, 130, 1000])
def test_chunks_past_a_rows_end_stay(L, act):
    """A prompt keeps the state before every chunk that has a token, and leaves the rest of a row's alone."""
    torch = require_gpu()
    log(f"chunks {L} {act}")
    lengths = [n for n in (L, 0, 1, 63, 64, 65, 128, 129, L - 1) if n <= L]
    op = GatedRecurrence(len(lengths), 70, act)
    x = torch.randn(len(lengths), L, 70, generator=torch.Generator().manual_seed(L)).to(op.tdtype).cuda()
    kept = op.new_chunk_states(L).fill_(float("nan"))
    op.prefill(x, x, x, lengths=torch.tensor(lengths, dtype=torch.int32).cuda(), chunk_states=kept)
    for b, n in enumerate(lengths):
        used = -(-n // hb.HM_RECURRENCE_CHUNK)
        assert torch.isfinite(kept[b, :used]).all() and torch.isnan(kept[b, used:]).all(), n
        assert used == 0 or not kept[b, 0].any()


def test_streams_by_their_handles():
    """A stream is given as torch's object or as its hipStream_t, the default one's 0 among them."""
    torch = require_gpu()
    log("handles of streams")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for user, (call, new) in _users(torch).items():
        x = new()
        want = call(x, None)
        torch.cuda.synchronize()
        for stream in (side, side.cuda_stream, 0, torch.cuda.default_stream().cuda_stream):
            got = call(x, stream)
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(got, want)), (user, stream)
