"""The timed cases' plain forms (perf/operators.py) against their definition in 64 bits: a quantizer's
codes and scales are exact, so they are compared for equality."""
import importlib.util
import os

import pytest
import torch

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "perf", "operators.py")


@pytest.fixture(scope="module")
def ops():
    spec = importlib.util.spec_from_file_location("operator_cases", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("rows,n", [(4096, 4096), (777, 11000), (2000, 129)])
def test_plain_rows_are_the_definition(ops, dtype, rows, n):
    g = torch.Generator(device="cuda").manual_seed(rows + n)
    x = torch.randn(rows, n, generator=g, device="cuda").to(dtype)
    q, d = ops._quantize(x)
    q64, d64 = ops._rows64(x)
    assert torch.equal(d.double(), d64[:, 0])
    assert torch.equal(q, q64)


@pytest.mark.parametrize("name", ["append_prompts", "append_decode"])
def test_plain_append_is_the_definition(ops, name):
    """Scales for equality; a value read back is scale * code rounded to binary32 and to bfloat16 (half
    steps of 2^-24 and 2^-8), where another code would be a part 1/127 of it off at least."""
    case = next(c for c in ops.listed() if c["name"] == name)
    got, want = ops.run(ops.prepare(case, 5)), ops.exact(case, 5)
    for s in ("k_scales", "v_scales"):
        assert torch.equal(got[s].double(), want[s])
    for s in ("k", "v"):
        off = (got[s].double() - want[s]).abs()
        assert (off <= (2.0 ** -8 + 2.0 ** -23) * want[s].abs()).all(), int((off > 2.0 ** -7 * want[s].abs()).sum())
