"""The bounded waits of the int8 product and attention, made to run out: a build of these kernels whose
waits give up at once.  Every call returns, says IQQ_FLAG_WAIT_TIMEOUT, and leaves the device to the next
call, which is right.  (What a CTA has under way itself it still waits for in full, and nothing that did
not arrive is used as an address, so no access depends on the waits that give up.)"""
import ctypes
import glob
import importlib.util
import os
import subprocess

import pytest
import torch

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def iqq():
    import post_weight_quantization_rowwise_b200 as m
    return m


@pytest.fixture(scope="module")
def short(iqq, tmp_path_factory):
    spec = importlib.util.spec_from_file_location(
        "_iqq_lib_build", os.path.join(ROOT, "post_weight_quantization_rowwise_b200", "build.py"))
    b = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(b)
    if not os.path.exists(b.nvcc()):
        pytest.skip("needs nvcc")
    to = str(tmp_path_factory.mktemp("short_waits"))
    names = ["abi.cu", "sm100.cu"] + [os.path.basename(p) for w in ("i8_*", "kv8_*") for p in glob.glob(os.path.join(b.CSRC, w + ".cu"))]
    flags = [f for f in b.NVCC_FLAGS if f != "-shared"] + ["-DIQQ_WAIT_CLOCKS=0", "-I", b.INCLUDE, "-I", b.CSRC]
    runs = [subprocess.Popen([b.nvcc(), *flags, "-c", os.path.join(b.CSRC, n), "-o", os.path.join(to, n + ".o")]) for n in names]
    assert [r.wait() for r in runs] == [0] * len(runs)
    lib = os.path.join(to, "libiqq_short.so")
    subprocess.run([b.nvcc(), *b.NVCC_FLAGS, "-o", lib, *[os.path.join(to, n + ".o") for n in names]], check=True)
    return ctypes.CDLL(lib)


@pytest.fixture
def both(iqq, short, monkeypatch):
    """call(f): f(flags) with the short waits, which has to time out; then f(flags) with the library's."""
    def call(f):
        flags = torch.zeros(1, dtype=torch.int32, device="cuda")
        with monkeypatch.context() as mp:
            for name in ("iqq_gemm_i8", "iqq_kv8_attention", "iqq_kv8_attention_workspace_bytes"):
                own, fn = getattr(iqq._lib, name), getattr(short, name)
                fn.argtypes, fn.restype = own.argtypes, own.restype
                mp.setitem(iqq._lib.__dict__, name, fn)
            for _ in range(3):
                f(flags)
            torch.cuda.synchronize()
        assert int(flags.item()) == iqq.FLAG_WAIT_TIMEOUT
        flags.zero_()
        out = f(flags)
        assert int(flags.item()) == 0
        return out
    return call


@pytest.mark.parametrize("n_tok,n_out,k", [(1, 128, 128), (1, 4096, 4096), (16, 2000, 4096), (100, 300, 5000),
                                           (300, 259, 1000), (1100, 5000, 2000)])
def test_product(iqq, both, n_tok, n_out, k):
    g = torch.Generator(device="cuda").manual_seed(k)
    a, w = (torch.randint(-127, 128, (n, (k + 15) // 16 * 16), generator=g, device="cuda").to(torch.int8)[:, :k]
            for n in (n_tok, n_out))
    da, dw = torch.ones(n_tok, device="cuda"), torch.ones(n_out, device="cuda")
    y = both(lambda flags: iqq.gemm_i8(a, da, w, dw, flags=flags))
    assert torch.equal(y, (a.double() @ w.double().t()).float())


def _attention(iqq, both, dim, lens, new, heads):
    page, n = 64, sum(-(-m // 64) for m in lens)
    g = torch.Generator(device="cuda").manual_seed(dim)
    codes = [torch.randint(-127, 128, (n, 1, page, dim), generator=g, device="cuda").to(torch.int8) for _ in range(2)]
    scales = [torch.rand(n, 1, generator=g, device="cuda") * 0.02 for _ in range(2)]
    cache = iqq.Kv8Cache(*codes, *scales)
    width, at, rows = max(-(-m // page) for m in lens), 0, []
    for m in lens:
        rows.append([at + i if i < -(-m // page) else 0 for i in range(width)])
        at += -(-m // page)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    args = (i32(rows), i32(lens), i32([sum(new[:b]) for b in range(len(new) + 1)]))
    q = torch.randn(sum(new), heads, dim, generator=g, device="cuda").to(torch.bfloat16)
    want = iqq.kv8_attention(cache, q, *args)
    out = both(lambda flags: iqq.kv8_attention(cache, q, *args, flags=flags))
    assert torch.equal(out, want)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("lens,new,heads", [([300], [300], 2), ([9000], [100], 4), ([700] * 12, [600] * 12, 8)])
def test_prompts(iqq, both, dim, lens, new, heads):
    _attention(iqq, both, dim, lens, new, heads)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("lens,new,heads", [([40], [1], 1), ([600, 30], [1, 1], 4), ([9000, 200], [1, 1], 8),
                                            ([3000] * 40, [3] * 40, 4)])
def test_tokens(iqq, both, dim, lens, new, heads):
    _attention(iqq, both, dim, lens, new, heads)
