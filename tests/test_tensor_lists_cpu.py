"""The binding's readers of tensor lists: the native one, and the one in Python that the calls on many tensors fall back
to, so that gradient norm, clipping and the step need no compiler beside the library."""
import sys
import types
import warnings

import pytest
import torch

import chunk_wise_weight_amd as ttt
from chunk_wise_weight_amd import binding, build


@pytest.fixture
def fresh(monkeypatch):
    """The choice of reader made anew, and undone."""
    monkeypatch.setattr(binding, "_read", None)


def native():
    return pytest.importorskip("chunk_wise_weight_amd._tensor_lists").read


def test_the_native_reader_is_built_and_taken(fresh):
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        assert binding._reader() is native()


LISTS = [
    [],
    [torch.zeros(3)],
    [torch.zeros(3, 4), torch.zeros(0, dtype=torch.bfloat16), torch.zeros((), dtype=torch.uint8)],
    [torch.zeros(3, 4).T, torch.zeros(5, dtype=torch.int16)],
    [torch.zeros(2, dtype=torch.float64), torch.zeros(2, dtype=torch.int64), torch.nn.Parameter(torch.zeros(7))],
    [torch.zeros(2).to_sparse(), torch.zeros(1, 1).expand(4, 4)],
]


@pytest.mark.parametrize("ts", LISTS)
def test_both_readers_give_the_same(ts):
    for device in (-1, 0):
        assert binding._read_python(ts, "grads", device) == native()(ts, "grads", device)


@pytest.mark.parametrize("bad", [None, 3, "x", [torch.zeros(1)]])
def test_both_readers_name_what_is_no_tensor(bad):
    for read in (binding._read_python, native()):
        with pytest.raises(TypeError, match=f"copies must be tensors, got {type(bad).__name__}"):
            read([torch.zeros(2), bad], "copies", 0)


def test_calls_work_without_the_native_reader(fresh, monkeypatch):
    monkeypatch.setitem(sys.modules, "chunk_wise_weight_amd._tensor_lists", None)
    monkeypatch.delattr(ttt, "_tensor_lists", raising=False)
    x = torch.zeros(4)
    with pytest.warns(RuntimeWarning, match="read in Python"):
        assert binding._reader() is binding._read_python
    with warnings.catch_warnings():
        warnings.simplefilter("error")  # once is enough
        for call in (lambda: ttt.ttt_grad_norm([x]), lambda: ttt.ttt_clip_grads([x], 1.0),
                     lambda: ttt.ttt_adamw([x], [x], [x], [x], 1, 1e-3)):
            with pytest.raises(ValueError, match="device tensors"):
                call()
        with pytest.raises(TypeError, match="grads must be tensors"):
            ttt.ttt_grad_norm([x, None])


@pytest.mark.parametrize("attributes", [{"built_for": "torch 1.0, Python 2.7"}, {}])
def test_one_built_for_another_torch_is_not_used(fresh, monkeypatch, attributes):
    other = types.ModuleType("chunk_wise_weight_amd._tensor_lists")
    other.read = None
    for k, v in attributes.items():
        setattr(other, k, v)
    monkeypatch.setitem(sys.modules, other.__name__, other)
    monkeypatch.setattr(ttt, "_tensor_lists", other, raising=False)
    with pytest.warns(RuntimeWarning, match="built for"):
        assert binding._reader() is binding._read_python


@pytest.mark.parametrize("cxx", ["/nowhere/g++", "false"])
def test_the_build_goes_on_without_a_host_compiler(monkeypatch, tmp_path, cxx):
    left = tmp_path / "_tensor_lists.so"
    left.write_bytes(b"of an earlier build")
    monkeypatch.setattr(build, "LISTS", str(left))
    monkeypatch.setenv("CXX", cxx)
    with pytest.warns(RuntimeWarning, match="read in Python"):
        assert build._build_lists(False) is False
    assert not left.exists()


def test_every_list_names_what_is_no_tensor_in_it():
    """Also tops, whose shapes are looked at."""
    call = binding._Call(torch.device("cpu"), None)
    like = types.SimpleNamespace(numel=b"", n=0)
    with pytest.raises(TypeError, match="tops must be tensors, got NoneType"):
        binding._tops(call, [None], like)
