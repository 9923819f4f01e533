"""Host threads that call the operators around the LM head at the same time, each
on a stream of its own with buffers of its own."""
import threading

import pytest
import torch

import entropy_active_span_gb300 as eas

pytestmark = pytest.mark.gpu


def _norms(H, seed, rounds, errors, barrier):
    """`rounds` forward and backward calls; the outputs of all must be alike."""
    try:
        g = torch.Generator().manual_seed(seed)
        x, r, ds = (torch.randn(6, H, generator=g).bfloat16().cuda() for _ in range(3))
        w = torch.ones(H, dtype=torch.bfloat16, device="cuda")
        out = (torch.empty_like(x), torch.empty(6, H, dtype=torch.uint8, device="cuda"),
               torch.empty(6, device="cuda"), torch.empty_like(x))
        dx, dw = torch.empty_like(x), torch.empty(H, device="cuda")
        ws = eas.workspace(eas.rmsnorm_bwd_workspace_size(6, H), "cuda")
        torch.cuda.synchronize()
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            def once():
                eas.rmsnorm_fwd(x, w, 1e-6, r, want_e4m3=True, out=out)
                eas.rmsnorm_bwd(x, r, w, 1e-6, ds, ws=ws, dx=dx, dweight=dw)
            once()
            want = [t.clone() for t in (*out, dx, dw)]
            barrier.wait(60)
            for i in range(rounds):
                once()
                if i % 250 == 249:
                    assert all(torch.equal(a, b) for a, b in zip((*out, dx, dw), want))
        stream.synchronize()
    except BaseException as e:  # noqa: B036 - handed to the thread that started this one
        errors.append(e)
        barrier.abort()


def test_rows_of_two_widths_at_once():
    """4096 and 8192 columns run the same kernels with different amounts of shared
    memory: what one thread's launch needs must not depend on the other's."""
    errors, barrier = [], threading.Barrier(4)
    threads = [threading.Thread(target=_norms, args=(H, i, 4000, errors, barrier))
               for i, H in enumerate((4096, 8192, 4096, 8192))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
