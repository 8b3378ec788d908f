"""What the wrappers of the few-token operators hand to the library, and what they refuse (CPU
only: the library's calls are recorded, not made; only its size calls run)."""
import os

import pytest
import torch

from dropless_token_routing_gb300 import builder as B

if not os.path.exists(B.LIB):
    B.build()

from dropless_token_routing_gb300 import _native as N  # noqa: E402
from dropless_token_routing_gb300 import api as A  # noqa: E402


class Stream:
    cuda_stream = 0


ST = Stream()
DEV = "cpu:0"   # the layers' device in these tests


class Recorder:
    """Stands in for the library: size calls go to it, all others are recorded and succeed."""

    def __init__(self, lib):
        self.lib, self.calls = lib, []

    def __getattr__(self, name):
        if name.endswith("_workspace_bytes"):
            return getattr(self.lib, name)

        def call(*args):
            # structures change between calls: their values now
            values = [getattr(a, "_obj", a) for a in args]
            values = [{f: getattr(v, f) for f, _ in v._fields_} if hasattr(v, "_fields_") else v for v in values]
            self.calls.append((name, values))
            return 0

        return call

    def last(self, name):
        got = [values for n, values in self.calls if n == name]
        return got[-1]


@pytest.fixture
def lib(monkeypatch):
    rec = Recorder(N.lib())
    monkeypatch.setattr(N, "lib", lambda: rec)
    return rec


def linear(N_=32, K=64, rows=8, dtype=torch.float32, **kw):
    return A.Linear(torch.zeros(N_, K, dtype=dtype), None, max_rows=rows, device=DEV, stream=ST, **kw)


# ------------------------------------------------------------------ rows that lie on one another
def test_linear_refuses_rows_closer_than_their_width(lib):
    """A broadcast row (stride 0) is no matrix of M rows: the library would take stride 0 for
    the default and read M - 1 rows past its end."""
    M, n, k = 4, 32, 64
    lin = linear()
    x, r, dy = torch.zeros(M, k), torch.zeros(M, n), torch.zeros(M, n)
    row = torch.zeros(n).expand(M, n)
    near = torch.zeros(M * n).as_strided((M, n), (n - 1, 1))   # rows overlap by one element
    lin.forward(x, residual=r, save=True, stream=ST)
    for bad in (row, near):
        with pytest.raises(ValueError):
            lin.forward(x, residual=bad, stream=ST)
        with pytest.raises(ValueError):
            lin.forward(x, out=bad, stream=ST)
    with pytest.raises(ValueError):
        lin.forward(torch.zeros(k).expand(M, k), stream=ST)
    lin.forward(x, save=True, stream=ST)
    with pytest.raises(ValueError):
        lin.backward(torch.zeros(M, n).sum(0).expand(M, n), stream=ST)
    lin.backward(dy, stream=ST)
    with pytest.raises(ValueError):
        A.Linear(torch.zeros(k).expand(n, k), None, max_rows=M, device=DEV, stream=ST)
    # a width of one element: its rows overlap with stride 0 alone
    one = A.Linear(torch.zeros(1, 1), None, max_rows=M, device=DEV, stream=ST)
    with pytest.raises(ValueError):
        one.forward(torch.zeros(1, 1).expand(M, 1), stream=ST)
    one.forward(torch.zeros(M, 1), stream=ST)


def test_linear_accepts_one_row_of_any_stride(lib):
    lin = linear()
    lin.forward(torch.zeros(64).expand(1, 64), residual=torch.zeros(32).expand(1, 32), stream=ST)
    dims = lib.last("moe_linear_fwd")[4]
    assert dims["M"] == 1 and dims["ld_x"] in (0, 64) and dims["ld_res"] in (0, 32)
