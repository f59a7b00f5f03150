"""The linear losses' workspace is exactly what the size call says: one byte less is
refused before anything runs, that much is enough, and nothing past it is touched."""
import numpy as np
import pytest
import torch

from tests.gpu_util import bits

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - CPU container
    pytest.skip("needs a GPU", allow_module_level=True)

import gemm_collective_gb300 as fcc  # noqa: E402
from tests.test_gpu_losses import Case  # noqa: E402

GUARD = 4 << 20


@pytest.mark.parametrize("kw", [dict(), dict(chunks=3), dict(max_ctas=5), dict(max_ctas=11, chunks=2),
                                dict(cta_pair=1), dict(cta_pair=2), dict(max_ctas=1)])
@pytest.mark.parametrize("R,T,V,D,K", [(1, 1, 1, 8, 0), (2, 45, 602, 72, 0), (2, 300, 1554, 328, 0),
                                       (1, 1100, 700, 1160, 7), (1, 33, 5000, 264, 200),
                                       (8, 129, 2056, 96, 1), (1, 20, 900, 520, 3)])
def test_the_stated_workspace_is_enough_and_needed(R, T, V, D, K, kw):
    c = Case(R, T, V, D, K=K, smoothing=0.0 if K else 0.1)
    loss, lse = c.forward()
    want = [bits(x) for x in (*loss, *lse)]
    for grad in (False, True):
        plain = fcc.make_opts(**kw)
        size = fcc.fcc_linear_loss_workspace_size(R, T, V, D, K, grad, plain)
        buf = torch.full((size + GUARD,), 0xA5, dtype=torch.uint8, device="cuda")

        def call(n):
            o = fcc.make_opts(workspace=buf, workspace_bytes=n, **kw)
            return c.backward(lse, o) if grad else c.forward(o)

        with pytest.raises(fcc.FccError) as e:
            call(size - 1)
        assert e.value.status == fcc.FCC_ERR_WORKSPACE
        assert (buf == 0xA5).all()
        got = call(size)
        torch.cuda.synchronize()
        assert (buf[size:] == 0xA5).all()
        if grad:
            ref = c.backward(lse, plain)
        else:
            ref = c.forward(plain)
            if not kw:
                for a, b in zip(want, [bits(x) for x in (*got[0], *got[1])]):
                    assert np.array_equal(a, b)
        for xs, ys in zip(got, ref):
            for x, y in zip(xs, ys):
                assert np.array_equal(bits(x), bits(y))
