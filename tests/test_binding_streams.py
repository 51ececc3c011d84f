"""The binding's `stream=` argument, on the host: what a wrapper allocates for a call on a
given stream comes from that stream's pool."""

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


def test_memory_belongs_to_the_given_stream(wq, monkeypatch):
    """Allocated with it current; a result is marked as used on the caller's stream."""
    current = ["caller"]

    @contextlib.contextmanager
    def stream(s):
        current.append(s)
        yield
        current.pop()

    def alloc(n, tuples=False):
        blocks = tuple(Block(current[-1]) for _ in range(n))
        return blocks + (None,) if tuples else blocks[0]

    monkeypatch.setattr(wq.torch.cuda, "stream", stream)
    monkeypatch.setattr(wq.torch.cuda, "current_stream", lambda device=None: current[-1])
    for make, used in ((wq._scratch, []), (wq._result, ["caller"])):
        one = make("side", alloc, 1)
        assert one.stream == "side" and one.used_on == used
        for t in make("side", alloc, 3, tuples=True)[:3]:
            assert t.stream == "side" and t.used_on == used
        one = make(None, alloc, 1)
        assert one.stream == "caller" and one.used_on == []
    assert current == ["caller"]


def test_no_wrapper_with_a_stream_allocates_past_it(wq):
    """Every allocation in a function that takes `stream` goes through the two."""
    with open(wq.__file__) as f:
        tree = ast.parse(f.read())
    checked = 0
    for fn in tree.body:
        if not isinstance(fn, ast.FunctionDef) or fn.name in ("_scratch", "_result", "_stream") or \
                "stream" not in [a.arg for a in fn.args.args]:
            continue
        checked += 1
        for call in ast.walk(fn):
            if isinstance(call, ast.Call):
                name = call.func.attr if isinstance(call.func, ast.Attribute) else call.func.id
                assert not name.startswith(("empty", "zeros", "new_", "alloc_")) and \
                    not name.endswith("workspace"), (fn.name, name, call.lineno)
    assert checked >= 25


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
