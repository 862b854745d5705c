"""Where the tensors that a call makes itself come from, without a GPU."""
import ast
import types

import pytest

torch = pytest.importorskip("torch")

import rank_sum_residual_gb300 as farn  # noqa: E402

MAKERS = {"empty", "empty_like", "empty_strided", "new_empty", "zeros", "zeros_like", "new_zeros",
          "full", "ones"}


def test_calls_make_tensors_in_one_place():
    """Every operator takes a stream, so none asks torch for memory of the current
    one: they all go through _new.  (kv_cache is no call on a stream.)"""
    tree = ast.parse(open(farn.__file__).read())
    found = {}
    for f in ast.walk(tree):
        if isinstance(f, ast.FunctionDef):
            for n in ast.walk(f):
                if isinstance(n, ast.Call) and isinstance(n.func, ast.Attribute) and \
                        n.func.attr in MAKERS:
                    found.setdefault(f.name, []).append(n.lineno)
    assert set(found) == {"_new", "_new_elsewhere", "kv_cache"}, found


class Stream:
    def __init__(self, cuda_stream, device="dev"):
        self.cuda_stream, self.device = cuda_stream, device


class Tensor:
    def __init__(self, made_on):
        self.made_on, self.used_on = made_on, []

    def record_stream(self, s):
        self.used_on.append(s.cuda_stream)


@pytest.fixture
def fake(monkeypatch):
    """torch with streams that are only remembered; stream 7 is the current one, and
    device 3."""
    t = types.SimpleNamespace(now=Stream(7), index=3, full=False)

    def set_stream(s):
        t.now, t.index = s, 0

    def empty(shape, dtype, device):
        if t.full:
            raise MemoryError
        return Tensor(t.now.cuda_stream)
    t.empty = empty
    t.cuda = types.SimpleNamespace(
        Stream=Stream, ExternalStream=Stream, set_stream=set_stream,
        current_stream=lambda device: t.now, current_device=lambda: t.index,
        set_device=lambda i: setattr(t, "index", i))
    monkeypatch.setattr(farn, "_torch", t)
    return t


@pytest.mark.parametrize("stream,made,used", [
    (None, 7, []), (Stream(7), 7, []), (Stream(9), 9, [7]),
    (types.SimpleNamespace(cuda_stream=9), 9, [7])])
def test_memory_of_the_calls_stream(fake, stream, made, used):
    new = farn._new(stream, "dev", ((2, 3), "a"), ((4,), "b"))
    assert [t.made_on for t in new] == [made] * 2
    assert [t.used_on for t in new] == [used] * 2
    work, = farn._new(stream, "dev", (8, "a"), returned=False)      # used on `stream` alone
    assert work.made_on == made and work.used_on == []
    assert fake.now.cuda_stream == 7 and fake.index == 3


def test_nothing_stays_switched(fake):
    with pytest.raises(ValueError, match="the stream is on other"):
        farn._new(Stream(9, "other"), "dev", (8, "a"))
    fake.full = True
    with pytest.raises(MemoryError):
        farn._new(Stream(9), "dev", (8, "a"))
    assert fake.now.cuda_stream == 7 and fake.index == 3
