"""The operators' calls run on their tensors' device, whichever is current (on the
host, with torch's and the library's parts replaced)."""
import contextlib
import re
import types

import pytest

from speculative_decoding_verification_83_gb300 import operators as ops

torch = pytest.importorskip("torch")


class Cuda:
    def __init__(self, current):
        self.current, self.made = current, []

    def current_device(self):
        return self.current

    @contextlib.contextmanager
    def device(self, d):
        before, self.current = self.current, d.index
        self.made.append(d.index)
        yield
        self.current = before


@pytest.mark.parametrize("current,index", [(0, 0), (1, 1), (0, 1), (1, 0)])
def test_calls_run_on_the_tensors_device(monkeypatch, current, index):
    cuda, seen = Cuda(current), []
    monkeypatch.setattr(ops, "_modules", [types.SimpleNamespace(cuda=cuda), None])
    ops._call(torch.device("cuda", index), lambda *a: seen.append((cuda.current, a)) or 0, 7, 8)
    assert seen == [(index, (7, 8))]
    assert cuda.current == current and cuda.made == ([] if current == index else [index])


def test_every_launch_goes_through_it():
    with open(ops.__file__) as f:
        s = f.read()
    launches = re.findall(r"(\w+\()?(?:dev, )?_library\(\)\.dflash_(\w+)", s)
    names = {"kv_append", "paged_attention", "distill_loss", "distill_grad", "distill_loss_grad"}
    assert {n for c, n in launches if c == "_call("} == names
    assert not [n for c, n in launches if c != "_call(" and n in names]
