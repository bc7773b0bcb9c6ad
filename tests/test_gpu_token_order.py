"""Token streams where CUDA streams, other streams' pages and unusual rows meet (needs a
GB300). Tolerances: see test_gpu_tokens."""

import numpy as np
import pytest
import torch

from oracle.tokens import causal_attend_fp64

from .test_gpu_tokens import SCALE, Pool, _built, f64, stored, tolerance   # noqa: F401 (_built: a fixture)

pytestmark = pytest.mark.gpu


def busy(seconds=0.05):
    """Finite work on the current stream."""
    torch.cuda._sleep(int(seconds * 1.5e9))


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
def test_a_stream_opened_behind_a_busy_default_stream(fp8):
    """Opened while the default stream has work to do, and used on a side stream at once:
    the pages and the joined splits are right before and after that work ends."""
    side, done = torch.cuda.Stream(), torch.cuda.Event()
    for waits in (0.0, 0.1):                     # the first turn loads the kernels
        p = Pool(400, 16, 2, fp8)
        torch.cuda.synchronize()
        for _ in range(2):                       # a handle's first open lays out its workspace, too
            busy(waits)
            done.record()
            sid = p.open()
            with torch.cuda.stream(side):
                batch = p.cache.token_batch([sid], [2000])
                k, v, q = p.rows(2000, 2), p.rows(2000, 2), p.rows(1, 4)
                p.ora.append([sid], [2000])
                p.cache.append_tokens(batch, k, v)
                out = p.cache.attend_tokens(p.cache.token_batch([sid], [1]), q)
                early = out.cpu()
            assert waits == 0 or not done.query(), "the default stream was to be busy meanwhile"
            kk, vv, qq = stored(k, fp8), stored(v, fp8), f64(q)
            ref = causal_attend_fp64(qq, kk, vv, 1999, 0, 0, SCALE)
            assert (np.abs(f64(early) - ref) <= tolerance(qq, kk, vv, ref, 1999, 0, 0, SCALE)).all()
            torch.cuda.synchronize()
            p.check_state(range(sid + 1))
            assert torch.equal(p.cache.attend_tokens(p.cache.token_batch([sid], [1]), q), out)
            torch.cuda.synchronize()
        p.cache.sync()
        p.cache.close()
