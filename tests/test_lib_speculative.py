"""favor_decode_tree / favor_decode_extend / favor_decode_verify on the CPU: argument errors are answered
on the host before any CUDA call, by the library and by the binding (no compute call runs here)."""

import ctypes

import pytest
import torch

from linear_attention_positive_b200 import api

P, ODD, NULL = ctypes.c_void_p(256), ctypes.c_void_p(258), None  # never dereferenced
INVALID, UNSUPPORTED, WORKSPACE = api.FAVOR_ERR_INVALID_ARG, api.FAVOR_ERR_UNSUPPORTED, api.FAVOR_ERR_WORKSPACE


def shape(*a):
    return ctypes.byref(api.make_shape(*a))


def swapped(args, i, x):
    return args[:i] + [x] + args[i + 1:]


BAD_SHAPES = [((0, 1, 4, 64, 256, 1), INVALID), ((1, 1, 0, 64, 256, 1), INVALID), ((1, 1, 4, 64, 256, 7), INVALID),
              ((1, 1, 4, 96, 256, 1), UNSUPPORTED), ((1, 1, 4, 64, 48, 0), UNSUPPORTED),
              ((1, 1, 4, 64, 288, 0), UNSUPPORTED), ((256, 256, 4, 64, 64, 0), UNSUPPORTED)]


def test_decode_tree_refusals(favor_lib):
    f = favor_lib.favor_decode_tree
    ok = [shape(2, 3, 8, 64, 256, api.FAVOR_BF16)] + [P] * 6 + [NULL, P, NULL]
    for i in (1, 2, 3, 4, 5, 6, 8):
        assert f(*swapped(ok, i, NULL)) == INVALID
    for i in (1, 2, 3, 4, 5, 6, 7, 8):
        assert f(*swapped(ok, i, ODD)) == INVALID
    for dims, st in BAD_SHAPES:
        assert f(*swapped(ok, 0, shape(*dims))) == st
    assert f(*swapped(ok, 0, shape(1, 1, api.FAVOR_TREE_MAX_NODES + 1, 64, 256, 1))) == UNSUPPORTED
    assert f(*swapped(ok, 0, NULL)) == INVALID


def test_decode_extend_refusals(favor_lib):
    f, size = favor_lib.favor_decode_extend, favor_lib.favor_decode_extend_workspace_size
    ok = [shape(2, 3, 8, 64, 256, api.FAVOR_BF16), P, P, P, P, 4, P, P, P, 1 << 30, NULL]
    for i in (1, 2, 3, 4, 7):
        assert f(*swapped(ok, i, NULL)) == INVALID  # 4: an index width without an index
    for i in (1, 2, 3, 4, 6, 7):
        assert f(*swapped(ok, i, ODD)) == INVALID
    assert f(*swapped(ok, 5, 0)) == INVALID and f(*swapped(ok, 5, -1)) == INVALID
    for dims, st in BAD_SHAPES:
        assert f(*swapped(ok, 0, shape(*dims))) == st
        assert size(shape(*dims), 0) == 0
    for bad in (NULL, ctypes.c_void_p(264)):
        assert f(*swapped(ok, 8, bad)) == WORKSPACE
    assert f(*swapped(ok, 9, 16)) == WORKSPACE
    assert size(NULL, 0) == 0 and size(shape(1, 1, 8, 64, 64, 1), -1) == 0


def test_decode_extend_workspace_follows_the_tokens_added(favor_lib):
    """A long prompt is cut into runs with partial states; an accepted path needs none of it, however
    many tokens the buffers hold."""
    size = favor_lib.favor_decode_extend_workspace_size
    long = shape(1, 16, 65536, 64, 256, api.FAVOR_BF16)
    assert size(long, 0) >= 2 * 16 * (64 * 256 + 2 * 256) * 4 and size(long, 0) % 256 == 0
    assert 0 < size(long, 9) <= 256


def test_decode_verify_refusals(favor_lib):
    f = favor_lib.favor_decode_verify

    def vs(*a):
        return ctypes.byref(api.VerifyShape(*a))

    ok = [vs(2, 8, 1000, api.FAVOR_F32), P, P, NULL, P, NULL, P, P, P, P, P, NULL]
    for i in (0, 1, 2, 4, 6, 7, 8, 9, 10):
        assert f(*swapped(ok, i, NULL)) == INVALID
    for i in (1, 2, 3, 4, 5, 6, 7, 8, 9, 10):
        assert f(*swapped(ok, i, ODD)) == INVALID
    for dims in ((0, 8, 1000, 0), (2, 0, 1000, 0), (2, 8, 0, 0), (2, 8, 1000, 5)):
        assert f(*swapped(ok, 0, vs(*dims))) == INVALID
    assert f(*swapped(ok, 0, vs(2, api.FAVOR_TREE_MAX_NODES + 1, 1000, 0))) == UNSUPPORTED
    assert f(*swapped(ok, 0, vs(65536, 8, 1000, 0))) == UNSUPPORTED


def test_binding_refuses_host_tensors(favor_lib):
    x = torch.zeros(1, 2, 4, 64)
    W, state, par = torch.zeros(64, 64), torch.zeros(2 * 66 * 64), torch.zeros(1, 4, dtype=torch.int32)
    for call in (lambda: api.decode_tree(x, x, x, W, state, par), lambda: api.decode_extend(x, x, W, state),
                 lambda: api.decode_verify(par, par, torch.zeros(1, 4, 10), torch.zeros(1, 4), torch.zeros(1))):
        with pytest.raises(api.FavorError) as e:
            call()
        assert e.value.status == INVALID


def test_extend_workspace_is_asked_for_on_the_tensors_device(favor_lib, monkeypatch):
    """The size follows the SM count of the current device, so it is asked for with the tensors' device
    current (stand-ins for the device switch and the library)."""
    current = [0]

    class Device:
        def __init__(self, index):
            self.index = index

        def __enter__(self):
            self.before, current[0] = current[0], self.index

        def __exit__(self, *_):
            current[0] = self.before

    class Library:
        @staticmethod
        def favor_decode_extend_workspace_size(shape, n_index):
            return 1000 + current[0]

    monkeypatch.setattr(torch.cuda, "device", Device)
    monkeypatch.setattr(api, "library", lambda: Library)
    dims = (1, 16, 4096, 64, 256, api.FAVOR_BF16)
    api._extend_workspace.cache_clear()
    try:
        assert [api._extend_workspace(i, 0, *dims) for i in (1, 0, 1)] == [1001, 1000, 1001]
    finally:
        api._extend_workspace.cache_clear()


def test_a_workspace_is_memory_of_the_tensors_device():
    """Its size counts in bytes whatever its type; one of another device is refused before any call."""
    cpu = torch.device("cpu")
    assert api._workspace_bytes(torch.empty(300, dtype=torch.float32), cpu) == 1200
    for bad, device in ((torch.empty(300), torch.device("cuda:0")), (torch.empty(300, device="meta"), cpu),
                        (torch.empty(20, 30).t(), cpu)):
        with pytest.raises(api.FavorError) as e:
            api._workspace_bytes(bad, device)
        assert e.value.status == INVALID


def test_decode_extend_refuses_token_counts_whose_runs_would_pass_32_bits(favor_lib):
    f, size, most = favor_lib.favor_decode_extend, favor_lib.favor_decode_extend_workspace_size, 1 << 30
    for dtype in (api.FAVOR_F32, api.FAVOR_BF16):
        few, many = shape(1, 1, 8, 64, 256, dtype), shape(1, 1, most + 1, 64, 256, dtype)
        assert size(few, most) > 0
        for n in (most + 1, 2**31 - 1):
            assert size(few, n) == 0
            assert f(few, P, P, P, P, n, P, P, P, 1 << 40, NULL) == UNSUPPORTED
        assert size(many, 0) == 0
        assert f(many, P, P, P, NULL, 0, P, P, P, 1 << 40, NULL) == UNSUPPORTED


def test_calls_run_with_the_tensors_device_current(monkeypatch):
    """On the tensors' device and its current stream, or the given one (stand-ins for CUDA)."""
    current, seen = [0], []

    class Device:
        def __init__(self, device):
            self.index = device.index

        def __enter__(self):
            self.before, current[0] = current[0], self.index

        def __exit__(self, *_):
            current[0] = self.before

    monkeypatch.setattr(torch.cuda, "device", Device)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda i: 100 + i, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: current[0], raising=False)

    def entry(*args):
        seen.append((current[0],) + args)
        return api.FAVOR_OK

    class Stream:
        cuda_stream = 77

    for index in (0, 1):
        api._launch("call", entry, torch.device("cuda", index), None, "a")
        api._launch("call", entry, torch.device("cuda", index), Stream, "b")
    assert seen == [(0, "a", 100), (0, "b", 77), (1, "a", 101), (1, "b", 77)]
    assert current == [0]


def test_a_stream_of_another_device_is_refused():
    class Stream:
        device = torch.device("cuda", 1)

    with pytest.raises(api.FavorError) as e:
        api._empty((4,), torch.float32, torch.device("cuda", 0), Stream)
    assert e.value.status == INVALID
