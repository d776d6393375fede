"""The Python binding without its extension: what only needs the C ABI works with
libkda.so alone.  The data pointers are fake and never dereferenced."""
import ctypes
import importlib.util
import os

import pytest

from gated_delta_rule_82_amd import kda

pytestmark = pytest.mark.skipif(not os.path.exists(kda.LIB_PATH), reason="libkda.so not built (run the build first)")


def binding(extension):
    """A copy of the binding that finds its extension at ``extension``."""
    spec = importlib.util.spec_from_file_location("kda_copy", kda.__file__)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    module.BINDING_PATH = extension
    return module


@pytest.mark.parametrize("what", ["missing", "broken"])
def test_c_abi_without_the_extension(tmp_path, what):
    path = str(tmp_path / "_kda_binding.so")
    if what == "broken":
        open(path, "w").write("not a library")
    copy = binding(path)
    assert copy.library().kda_abi_version() == kda.library().kda_abi_version()
    assert copy.status_string(copy.KDA_ERR_SHAPE) == kda.status_string(kda.KDA_ERR_SHAPE)
    assert copy.check_host([0, 2], [0], 2, 1) == copy.KDA_OK
    t = copy.raw_tensor(0x10000, copy.KDA_F32, (3,))
    assert copy.call_raw([t] * 11, copy.make_mode()) == copy.KDA_ERR_SHAPE
    assert copy.call_raw_gdr([t] * 11, copy.make_mode()) == copy.KDA_ERR_SHAPE
    assert copy.call_raw_verify([t] * 9) == copy.KDA_ERR_SHAPE


@pytest.mark.parametrize("what", ["missing", "broken"])
def test_call_path_without_the_extension(tmp_path, what):
    """The call path refuses what the extension refuses, and reaches the library."""
    path = str(tmp_path / "_kda_binding.so")
    if what == "broken":
        open(path, "w").write("not a library")
    copy = binding(path)
    copy.library()
    copy._load_native()
    assert copy._native is copy._described_call
    torch = pytest.importorskip("torch")
    x = torch.zeros(3)
    for tensors in ((x,) * 11, (None,) * 11, (3.0,) * 11):     # not on a GPU, not a tensor
        assert copy._native(copy._RECURRENCE, copy._ENTRY["kda_decode"], tensors, 0, 0, 0.0, 0.0, 0.0, 0, 0, 0) is None


def test_extension_loads_where_it_is_built():
    if not os.path.exists(kda.BINDING_PATH):
        pytest.skip("the extension is not built")
    copy = binding(kda.BINDING_PATH)
    copy.library()
    copy._load_native()
    assert copy._native is not copy._described_call


def test_entry_points_take_structs_and_check_their_types():
    """The entry points of library() take descriptors themselves, by reference or as
    pointers, and refuse a struct of another type."""
    lib = kda.library()
    t, mode = kda.raw_tensor(0x10000, kda.KDA_F32, (3,)), kda.make_mode()
    by_kind = {"kda_decode": [t] * 11 + [mode, None], "kda_prefill": [t] * 11 + [mode, 0, None],
               "kda_gdr_decode": [t] * 11 + [mode, None], "kda_gdr_prefill": [t] * 11 + [mode, None],
               "kda_decode_window": [t] * 11 + [kda.KdaReplay(), mode, None],
               "kda_decode_conv": [t, kda.KdaConv()] + [t] * 7 + [mode, None], "kda_verify": [t] * 9 + [None]}
    for name, args in by_kind.items():
        fn = getattr(lib, name)
        refs = [ctypes.byref(a) if isinstance(a, ctypes.Structure) else a for a in args]
        pointers = [ctypes.pointer(a) if isinstance(a, ctypes.Structure) else a for a in args]
        assert fn(*args) == fn(*refs) == fn(*pointers) < 0, name
        with pytest.raises(ctypes.ArgumentError):
            fn(*[ctypes.byref(mode)] * 2, *args[2:])
