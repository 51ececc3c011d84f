"""The binding on the host: a call with `stream=` is made with that stream current, so that
what the wrapper allocates comes from that stream's pool; and what needs no GPU."""

import ast
import contextlib
import subprocess
import sys

import pytest

from tests.conftest import ROOT


@pytest.fixture(scope="module")
def wq():
    from bit_weight_quantized_weights_b200 import build_lib
    build_lib.build()
    from bit_weight_quantized_weights_b200 import binding
    return binding


class Block:
    device = "cuda:0"

    def __init__(self, stream):
        self.stream, self.used_on = stream, []

    def record_stream(self, stream):
        self.used_on.append(stream)


def test_a_call_on_a_stream_is_made_with_it_current(wq, monkeypatch):
    """What it allocates is that stream's; its results are marked as used on the caller's."""
    current = ["caller"]

    @contextlib.contextmanager
    def stream(s):
        current.append(s)
        yield
        current.pop()

    def wrapper(n, tuples=False):
        blocks = tuple(Block(current[-1]) for _ in range(n))
        return blocks + (None,) if tuples else blocks[0]

    monkeypatch.setattr(wq.torch.cuda, "stream", stream)
    monkeypatch.setattr(wq.torch.cuda, "current_stream", lambda device=None: current[-1])
    results = [wq._on("side", wrapper, 1)] + list(wq._on("side", wrapper, 3, True)[:3])
    assert all(t.stream == "side" and t.used_on == ["caller"] for t in results)
    assert current == ["caller"]


def test_every_wrapper_with_a_stream_goes_on_it_first(wq):
    """Each begins with the same call of itself, with all its other arguments, on the stream."""
    with open(wq.__file__) as f:
        tree = ast.parse(f.read())
    checked = 0
    for fn in tree.body:
        if not isinstance(fn, ast.FunctionDef):
            continue
        names = [a.arg for a in fn.args.args]
        # (the error word's read allocates nothing)
        if "stream" not in names or fn.name in ("_on", "_stream", "wq_device_error"):
            continue
        checked += 1
        body = fn.body[1:] if ast.get_docstring(fn) is not None else fn.body
        rest = [n for n in names if n != "stream"]
        assert ast.unparse(body[0]) == "if stream is not None:\n    return _on(stream, %s)" % \
            ", ".join([fn.name] + rest), fn.name
    assert checked == 26


def test_host_calls_work_on_a_torch_without_cuda(wq):
    """Sizes, the codebook and refusals need neither a GPU nor torch's CUDA bindings."""
    code = ("import torch\n"
            "del torch._C._cuda_getCurrentRawStream\n"
            "from bit_weight_quantized_weights_b200 import binding as wq\n"
            "assert len(wq.wq_nf4_codebook()) == 16\n"
            "assert wq.wq_workspace_bytes(wq.WQ_OP_MX_GEMM, 4, 256, 512, 0, 2) > 0\n"
            "assert wq.lib.wq_kv_append(*[None] * 2, 0, -1, 1, 128, None, None, 1, None, None, 8, "
            "*[None] * 7) == wq.WQ_ERR_INVALID_ARG\n")
    subprocess.run([sys.executable, "-c", code], check=True, cwd=ROOT, timeout=300)
