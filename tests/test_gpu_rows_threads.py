"""The packed-row calls from host threads other than the main one, and after a launch that the
driver refuses."""
import ctypes
import threading

import pytest

from test_gpu_rows import BF16, F32, Batch, slm  # noqa: F401  (slm: the fixture)

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


def together(*jobs):
    """Run the jobs at once, a thread each; what they raise."""
    errors, start = [], threading.Barrier(len(jobs))

    def work(job):
        try:
            start.wait()
            job()
        except Exception as e:  # noqa: BLE001  (seen by the caller)
            errors.append(e)

    threads = [threading.Thread(target=work, args=(j,)) for j in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    return errors


@pytest.mark.parametrize("dtype,hd", [(BF16, 64), (BF16, 128), (F32, 64), (F32, 256)])
def test_the_first_call_of_a_host_thread(slm, dtype, hd):  # noqa: F811
    """A thread that has not used the GPU yet has no current context: each call makes its own."""
    b = Batch(dtype, 4, 2, hd, [30, 1], None, 16, seed=1)
    want, out, ws = b.out(), b.out(), b.workspace(slm)
    stream = torch.cuda.Stream()

    def append():
        slm.kv_append(b.k, b.v, b.k_cache, b.v_cache, b.page_table, b.row_start, None, b.status, stream=stream)

    def paged(o=out):
        slm.attention_paged(b.q, b.k_cache, b.v_cache, b.page_table, b.row_start, None, o, ws, b.status, stream=stream)

    def prompt():
        slm.attention_prompt(b.q, b.k, b.v, b.row_start, out, ws, b.status, stream=stream)

    torch.cuda.synchronize()
    assert not together(append)
    paged(want)
    torch.cuda.synchronize()
    for job in (paged, prompt):
        out.fill_(7.0)
        torch.cuda.synchronize()
        errors = together(job)
        assert not errors, errors
        assert torch.equal(out, want)
    assert int(b.status.item()) == 0


@pytest.mark.parametrize("dtype,hd", [(BF16, 64), (BF16, 128), (BF16, 256), (F32, 64), (F32, 128)])
@pytest.mark.parametrize("chunk", [1, 40])
def test_two_host_threads(slm, dtype, hd, chunk):  # noqa: F811
    """Batches of very different numbers of sequences (and so of shared memory) on the same
    kernel, a thread, a stream and a workspace each: every call succeeds, with the bits that it
    gives alone.  chunk: the sequences' new tokens (the CUDA-core tile follows them)."""
    few = Batch(dtype, 4, 2, hd, [chunk], [100], 16, seed=1)
    many = Batch(dtype, 4, 2, hd, [chunk] * 500, [i % 50 for i in range(500)], 16, seed=2)
    jobs, outs = [], []
    for b in (few, many):
        b.fill([n + c for n, c in zip(b.new, b.ctx)])
        out, ws, stream = b.out(), b.workspace(slm), torch.cuda.Stream()

        def call(b=b, out=out, ws=ws, stream=stream):
            slm.attention_paged(b.q, b.k_cache, b.v_cache, b.page_table, b.row_start, b.ctx_len, out, ws, b.status,
                                stream=stream)

        torch.cuda.synchronize()
        call()
        torch.cuda.synchronize()
        outs.append((b, out, out.clone()))
        jobs.append(lambda call=call: [call() for _ in range(1500)])
    errors = together(*jobs)
    assert not errors, errors
    for b, out, want in outs:
        assert torch.equal(out, want)
        assert int(b.status.item()) == 0


def test_a_refused_launch_is_not_held_against_the_next_call(slm):  # noqa: F811
    """The legacy stream takes no work while a blocking stream is captured: the packed-row calls
    say so, and calls that follow do not meet the error again."""
    try:
        rt = ctypes.CDLL("libcudart.so.13")
    except OSError:
        pytest.skip("no shared CUDA runtime to capture with")
    b = Batch(BF16, 4, 2, 64, [1], [30], 16, seed=3)
    b.fill([31])
    out, ws = b.out(), b.workspace(slm)
    q = torch.ones(1, 4, 64, device="cuda")
    kc, ref = torch.ones(1, 2, 8, 64, device="cuda"), torch.zeros(1, 4, 64, device="cuda")
    aws = torch.empty(slm.slm_attention_workspace_bytes(1, 4, 2, 64), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    calls = [lambda: slm.attention_paged(b.q, b.k_cache, b.v_cache, b.page_table, b.row_start, b.ctx_len, out, ws, b.status,
                                         stream=0),
             lambda: slm.kv_append(b.k, b.v, b.k_cache, b.v_cache, b.page_table, b.row_start, b.ctx_len, b.status, stream=0)]
    for call in calls:
        stream, graph = ctypes.c_void_p(), ctypes.c_void_p()
        assert rt.cudaStreamCreate(ctypes.byref(stream)) == 0
        assert rt.cudaStreamBeginCapture(stream, 2) == 0  # relaxed: only this stream's work is watched
        try:
            with pytest.raises(slm.SlmError, match="launch"):
                call()
        finally:
            rt.cudaStreamEndCapture(stream, ctypes.byref(graph))
            rt.cudaGetLastError()
            assert rt.cudaStreamDestroy(stream) == 0
        assert slm.attention_decode(q, kc, kc, [8], ref, aws, slm.SLM_F32) == 0, slm.slm_last_error(None)
        torch.cuda.synchronize()
        assert bool((ref == 1).all())
