"""Forms of attention scores and shared prefixes as far as no GPU is needed: the definitions on
facts outside them, and what the calls refuse before anything is launched."""

import ctypes
import os

import numpy as np
import pytest
import torch

from oracle import entries as E
from speculative_decoding_verification_07_gb300 import binding

OK, INVALID, UNSUPPORTED = binding.SV_OK, binding.SV_ERR_INVALID, binding.SV_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(binding.LIB_PATH):
        from speculative_decoding_verification_07_gb300 import build
        build.build()
    return binding.load_library()


# --------------------------------------------------------------------------- #
# definitions
# --------------------------------------------------------------------------- #
def test_forms_of_one_row():
    rng = np.random.default_rng(0)
    q, K, V = rng.standard_normal(8), rng.standard_normal((20, 8)), rng.standard_normal((20, 8))
    far, seen = np.arange(19, -1, -1), np.ones(20, bool)
    plain = E.attend(q, K, V, seen, 0.3)[0]
    none = E.attend_shaped(q, K, V, seen, 0.3, far)
    assert (none[0] == plain).all() and none[3] == 0
    # a cap far above the scores changes nothing (s^3 / (3 c^2)), one at 0 makes all keys weigh the same
    np.testing.assert_allclose(E.attend_shaped(q, K, V, seen, 0.3, far, softcap=1e4)[0], plain, atol=1e-7)
    np.testing.assert_allclose(E.attend_shaped(q, K, V, seen, 0.3, far, softcap=1e-9)[0], V.mean(0), atol=1e-7)
    # a steep slope leaves the nearest key, a window of one too
    np.testing.assert_allclose(E.attend_shaped(q, K, V, seen, 0.3, far, slope=60.0)[0], V[-1], atol=1e-12)
    assert (E.attend_shaped(q, K, V, seen, 0.3, far, window=1)[0] == V[-1]).all()
    # equal scores under a slope of ln 2: each key half of the one after it
    o = E.attend_shaped(np.zeros(8), K[:3], np.eye(8)[:3], seen[:3], 1.0, far[-3:], slope=np.log(2))[0]
    np.testing.assert_allclose(o[:3], np.array([1, 2, 4]) / 7)
    # what a row does not see takes no part, whatever it holds
    V[4] = np.nan
    seen[4] = False
    assert np.isfinite(E.attend_shaped(q, K, V, seen, 0.3, far, softcap=2.0, slope=0.1)[0]).all()
    assert not E.attend_shaped(q, K, V, np.zeros(20, bool), 0.3, far, window=5)[0].any()


def test_groups_of_hand_written_tables():
    t = [[7, 8, 9, 1], [7, 8, 9, 2], [7, 8, 3, 2], [7, 4, 3, 2], [5, 4, 3, 2], [5, 4, 3, 2]]
    length, members = E.prefix_groups(t, [8] * 6, 2, 1)   # 3, 2, 1, 0 and 4 blocks in common
    assert length.tolist() == [2, 2, 2, 2, 8, 8] and members.tolist() == [4, 0, 0, 0, 2, 0]
    length, members = E.prefix_groups(t, [8] * 6, 2, 4)
    assert length.tolist() == [4, 4, 4, 0, 8, 8] and members.tolist() == [3, 0, 0, 0, 2, 0]
    length, members = E.prefix_groups(t, [8, 5, 8, 8, 8, 3], 2, 4)  # blocks that both have filled
    assert length.tolist() == [4, 4, 4, 0, 0, 0] and members.tolist() == [3, 0, 0, 0, 0, 0]
    length, members = E.prefix_groups([[-1, 2], [-1, 2]], [4, 4], 2, 1)  # no block at all
    assert not length.any() and not members.any()


# --------------------------------------------------------------------------- #
# host checks of the C entry points: nothing is launched, so the pointers are numbers
# --------------------------------------------------------------------------- #
def attention_args(**changed):
    a = binding.SvAttentionArgs()
    a.B, a.R, a.Hq, a.dtype = 4, 3, 8, binding.SV_BF16
    a.q = a.out = 1 << 20
    a.q_stride[:] = a.out_stride[:] = [3 * 8 * 128, 8 * 128, 128]
    a.seq_len, a.scale = 1 << 20, 0.1
    c = a.cache
    c.data, c.block_table, c.layers, c.heads, c.head_dim = 1 << 20, 1 << 20, 1, 2, 128
    c.format, c.layer, c.num_blocks, c.block_size, c.max_blocks = binding.SV_KV_BF16, 0, 64, 16, 16
    for k, v in changed.items():
        setattr(a, k, v)
    return a


def size_of(lib, a):
    handle = ctypes.create_string_buffer(4096)  # a host struct; only the number of SMs is read
    ctypes.cast(handle, ctypes.POINTER(ctypes.c_int32))[1] = 152
    n = ctypes.c_size_t()
    return lib.sv_attention_workspace_size(handle, ctypes.byref(a), ctypes.byref(n)), n.value


def test_arguments_of_forms(lib):
    plain = size_of(lib, attention_args())
    assert plain[0] == OK
    for ok in (dict(softcap=30.0), dict(softcap=2.0 ** -60), dict(softcap=2.0 ** 60), dict(window=1), dict(window=2 ** 31 - 1),
               dict(slopes=1 << 20), dict(depth=1 << 20), dict(shared_len=1 << 20, shared_members=1 << 20)):
        code, n = size_of(lib, attention_args(**ok))
        assert code == OK and (n > plain[1]) == ("depth" not in ok)  # the list of items
    for bad in (dict(softcap=-1.0), dict(softcap=float("nan")), dict(softcap=float("inf")), dict(softcap=2.0 ** -61), dict(softcap=2.0 ** 61),
                dict(window=-1), dict(shared_len=1 << 20), dict(shared_members=1 << 20)):
        assert size_of(lib, attention_args(**bad))[0] == INVALID, bad


def test_arguments_of_groups(lib):
    assert lib.sv_prefix_groups(None, 1, None, None, 1, 16, 1, None, None, None) == INVALID
    handle = ctypes.create_string_buffer(4096)
    p = ctypes.c_void_p(1 << 20)
    for args in ((-1, p, p, 4, 16), (2, None, p, 4, 16), (2, p, None, 4, 16), (2, p, p, -1, 16), (2, p, p, 4, 0)):
        assert lib.sv_prefix_groups(handle, *args, 1, p, p, None) == INVALID, args
    assert lib.sv_prefix_groups(handle, 2, p, p, 4, 16, 1, None, p, None) == INVALID
    at = lambda n: ctypes.c_void_p((1 << 20) + n)  # noqa: E731
    for table, length, members in ((1024, 2048, 2048), (1024, 2048, 2052), (1024, 4, 2048), (1024, 2048, 0), (1024, 1052, 2048),
                                   (1024, 2048, 1020)):  # outputs over one another and over inputs
        assert lib.sv_prefix_groups(handle, 2, at(0), at(table), 4, 16, 1, at(length), at(members), None) == INVALID
    assert lib.sv_prefix_groups(handle, 0, None, None, 4, 16, 1, None, None, None) == OK  # nothing to do


def test_refusals_of_the_python_calls():
    c = binding._calls()
    t, z = torch.zeros(2, 3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    for table, least in ((t.long(), 1), (t.t(), 1), (z, 1), (t, 2 ** 40)):
        with pytest.raises(ValueError):
            c.prefix_groups(None, table, z, 16, least, None, None, 0)
    for length, members in ((z, None), (None, z)):
        with pytest.raises(ValueError, match="length and members"):
            c.prefix_groups(None, t, z, 16, 1, length, members, 0)
    with pytest.raises(TypeError):
        c.attention_forms(None)
