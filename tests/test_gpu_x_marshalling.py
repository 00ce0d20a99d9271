"""GPU: the torch forms of the 8-bit operators and the update: the same results
whether their calls are marshalled by the extension or in Python, on any stream
and from any thread."""
import pytest

import mixed_precision_matmul_gb300 as mpg
from mixed_precision_matmul_gb300 import fp8

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("m,n,k", [(1, 300, 256), (70, 129, 515), (300, 260, 640)])
@pytest.mark.parametrize("block", ["row", "tile"])
def test_python_form_is_the_extension_s(m, n, k, block, monkeypatch):
    import torch
    mpg.build()
    assert fp8._calls() is not None
    g = torch.Generator(device="cuda").manual_seed(m)
    x, w = (torch.randn(s, generator=g, device="cuda") for s in ((m, k), (n, k)))

    def run():
        q = mpg.fp8_quantize(x.bfloat16(), fmt="e5m2", transpose=True)
        wq, ws = mpg.fp8_quantize(w, block=block)
        y = [mpg.gemm_fp8(q[0], q[1], wq, ws, alpha=0.5, out_dtype=t) for t in (None, torch.float32, torch.float16)]
        odd = mpg.gemm_fp8(q[0][:, 1:k - 1], q[1], wq[:, 1:k - 1], ws)         # off 16 bytes: copied
        return [*q, wq, ws, *y, odd]
    one = run()
    monkeypatch.setattr(fp8, "_calls", lambda: None)
    for a, b in zip(one, run()):
        assert a.dtype == b.dtype and a.stride() == b.stride() and torch.equal(a.float(), b.float())


def chain(x, w, stream):
    import torch
    q, s = mpg.fp8_quantize(x, stream=stream)
    wq, ws = mpg.fp8_quantize(w, block="tile", stream=stream)
    y = mpg.gemm_fp8(q, s, wq, ws, out_dtype=torch.float32, stream=stream)
    return y, mpg.orthogonalize(y, out_dtype=torch.float32, stream=stream)


@pytest.mark.parametrize("kind", ["torch stream", "handle", "an object with the handle", "the default stream's handle"])
def test_streams_as_the_other_entry_points_take_them(kind):
    import torch
    mpg.build()
    g = torch.Generator(device="cuda").manual_seed(4)
    x, w = (torch.randn(s, generator=g, device="cuda") for s in ((40, 256), (96, 256)))
    want = chain(x, w, None)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()

    class Holder:
        cuda_stream = side.cuda_stream
    stream = {"torch stream": side, "handle": side.cuda_stream, "an object with the handle": Holder(),
              "the default stream's handle": 0}[kind]
    got = chain(x, w, stream)
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_tensors_on_the_host_are_refused_with_a_stream_too():
    import torch
    mpg.build()
    side = torch.cuda.Stream()
    x = torch.zeros((4, 256))
    a, s = x.to(torch.float8_e4m3fn), torch.zeros((4, 2))
    for call in (lambda: mpg.fp8_quantize(x, stream=side), lambda: mpg.gemm_fp8(a, s, a, s, stream=side),
                 lambda: mpg.orthogonalize(x, stream=side), lambda: mpg.fp8_quantize(x, stream=side.cuda_stream)):
        with pytest.raises(ValueError, match="CUDA"):
            call()


def test_workspaces_with_gaps_or_repeats_are_refused():
    """An expanded tensor's bytes are not there; one with gaps is not what its size says."""
    import torch
    mpg.build()
    x = torch.randn((70, 515), device="cuda")
    q, s = mpg.fp8_quantize(x)
    odd = q[:, 1:513]
    need = mpg.orthogonalize_workspace_size(70, 515)
    for ws in (torch.empty(1, dtype=torch.uint8, device="cuda").expand(1 << 22),
               torch.empty(1 << 23, dtype=torch.uint8, device="cuda")[::2]):
        assert ws.numel() >= need
        with pytest.raises(ValueError, match="contiguous"):
            mpg.orthogonalize(x, workspace=ws)
        with pytest.raises(ValueError, match="contiguous"):
            mpg.gemm_fp8(odd, s[:, :4], odd, s[:, :4], workspace=ws)


def test_calls_from_several_threads():
    import threading

    import torch
    mpg.build()
    g = torch.Generator(device="cuda").manual_seed(5)
    shapes = [(5, 300, 256), (70, 129, 640), (300, 260, 512), (33, 96, 1024)]
    data = [tuple(torch.randn(t, generator=g, device="cuda") for t in ((m, k), (n, k))) for m, n, k in shapes]
    want = [chain(x, w, None) for x, w in data]
    torch.cuda.synchronize()
    wrong = []

    def work(i):
        try:
            side = torch.cuda.Stream()
            for r in range(12):
                j = (i + r) % len(data)
                got = chain(*data[j], side)
                side.synchronize()
                if not all(torch.equal(a, b) for a, b in zip(got, want[j])):
                    wrong.append((i, r))
        except Exception as e:                                  # noqa: BLE001 (reported below)
            wrong.append((i, repr(e)))
    threads = [threading.Thread(target=work, args=(i,)) for i in range(8)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong
    assert mpg.device_status() == mpg.OK
