"""4-bit weights without a GPU: an object that names packed weights holds them, and the ways of
cutting a product are the ones that the GPU tests run."""
import copy
import ctypes
import io
import pickle
import random

import pytest
import torch

import expert_routed_ffn_softmax_b200 as moe
from expert_routed_ffn_softmax_b200 import _abi, build
from w4_cuts import CUTS


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _abi.load()


# ----------------------------------------------------------------------------- W4Weights
def packed(E=2, K=128, N=32, R=544):
    return torch.zeros((E, N // 16, K // 64, R), dtype=torch.uint8)


def test_weights_object_takes_its_own_layout(lib):
    for group, zeros, R in ((32, False, 576), (32, True, 608), (64, False, 544), (64, True, 560),
                            (128, False, 544), (128, True, 560)):
        w = moe.W4Weights(packed(R=R), 2, 128, 32, group, zeros)
        assert w.shape == (2, 128, 32) and w.flags == (_abi.MOE_FLAG_W4_ZEROS if zeros else 0)
        assert w.index == -1 and w.device.type == "cpu"


def test_weights_object_refuses_another_layout(lib):
    """What the kernels would read past, or misread: another size, type, layout or form."""
    good = (2, 128, 32, 64, False)
    bad = [
        (packed(), (3, 128, 32, 64, False)), (packed(), (2, 192, 32, 64, False)),
        (packed(), (2, 128, 48, 64, False)), (packed(), (2, 128, 32, 32, False)),
        (packed(), (2, 128, 32, 64, True)), (packed(R=560), good), (packed(E=1), good),
        (packed().flatten(), good), (packed()[:, :, :, :-16], good),
        (packed(E=4)[::2], good), (packed().transpose(1, 2), good),
        (torch.zeros(packed().numel() + 8, dtype=torch.uint8)[8:].view(packed().shape), good),
    ]
    for data, args in bad:
        with pytest.raises(ValueError):
            moe.W4Weights(data, *args)
    for data in (packed().to(torch.int8), packed().to(torch.float32), None, [0] * 16):
        with pytest.raises(TypeError):
            moe.W4Weights(data, *good)
    with pytest.raises(TypeError):
        moe.W4Weights(packed(), 2, 128, 32.0, 64, False)
    for args in ((2, 100, 32, 64, False), (2, 128, 24, 64, False), (2, 128, 32, 16, False),
                 (0, 128, 32, 64, False), (2, 1 << 20, 32, 64, False)):
        with pytest.raises(moe.MoEError):
            moe.W4Weights(packed(), *args)


def test_weights_object_stays_what_it_is(lib):
    w = moe.W4Weights(packed(), 2, 128, 32, 64, False)
    for name in ("data", "E", "K", "N", "group", "zeros", "flags", "index"):
        with pytest.raises(AttributeError):
            setattr(w, name, getattr(w, name))


def test_weights_object_through_files_and_copies(lib):
    """A copy and a restored object go through the same checks, so its device is its data's."""
    w = moe.W4Weights(packed(), 2, 128, 32, 64, False)
    w.data[0, 0, 0, 0] = 7
    buf = io.BytesIO()
    torch.save(w, buf)
    buf.seek(0)
    for c in (copy.copy(w), copy.deepcopy(w), pickle.loads(pickle.dumps(w)),
              torch.load(buf, weights_only=False)):
        assert c.shape == w.shape and c.group == 64 and c.zeros is False and torch.equal(c.data, w.data)
        assert c.index == c.data.get_device()
    fn, args = w.__reduce__()
    with pytest.raises(ValueError):
        fn(args[0][:1], *args[1:])


def test_weights_object_saved_as_plain_slots(lib):
    """The state that a pickle of plain slots holds; a device number in it is not believed."""
    w = moe.W4Weights(packed(), 2, 128, 32, 64, False)
    slots = {n: getattr(w, n) for n in ("data", "E", "K", "N", "group", "zeros", "flags")}
    c = moe.W4Weights.__new__(moe.W4Weights)
    c.__setstate__((None, {**slots, "index": 3}))
    assert c.shape == w.shape and c.index == -1 and c.data is w.data
    with pytest.raises(ValueError):
        moe.W4Weights.__new__(moe.W4Weights).__setstate__((None, {**slots, "group": 32, "index": 0}))


def test_weights_on_the_host_are_refused_by_the_calls(lib):
    with pytest.raises(TypeError, match="CUDA"):
        moe.w4_dequantize(moe.W4Weights(packed(), 2, 128, 32, 64, False))


# ----------------------------------------------------------------------------- cuts
def cut_of(lib, geglu, T, K, N, group, zeros, sms=148):
    cut = (ctypes.c_int * 6)()
    rc = lib.moe_debug_w4_cut(T, K, N, group, _abi.MOE_FLAG_W4_ZEROS if zeros else 0, geglu, sms, cut)
    assert rc == 0
    cluster, strips, units, step, frag, steal = cut
    # every strip is in a unit and every block in a chunk, with nothing left over
    per = strips // 2 if geglu else strips
    assert (units - 1) * per < N // 16 <= units * per and cluster <= K // 64
    assert 1 <= step <= -(-(K // 64) // cluster)
    return geglu, cluster, strips, frag, steal


def test_listed_cuts_are_the_ones_taken(lib):
    for row in CUTS:
        assert cut_of(lib, row[0], *row[5:]) == row[:5], row
    assert len({row[:5] for row in CUTS}) == len(CUTS)


def test_no_cut_is_taken_that_is_not_listed(lib):
    rng, listed = random.Random(3), {row[:5] for row in CUTS}
    for _ in range(20000):
        geglu = rng.random() < 0.4
        N = 64 * int(2 ** rng.uniform(0, 7)) if geglu else 16 * int(2 ** rng.uniform(0, 16))
        shape = (rng.randint(1, 16), 64 * int(2 ** rng.uniform(0, 8)), N, rng.choice((32, 64, 128)),
                 rng.random() < 0.5)
        assert cut_of(lib, int(geglu), *shape) in listed, shape


def test_cut_query_refuses(lib):
    f, out = lib.moe_debug_w4_cut, (ctypes.c_int * 6)()
    assert f(8, 128, 64, 64, 0, 0, 148, None) == _abi.MOE_ERR_INVALID_ARG
    assert f(8, 128, 64, 48, 0, 0, 148, out) == _abi.MOE_ERR_INVALID_ARG
    assert f(8, 128, 64, 64, 1, 0, 148, out) == _abi.MOE_ERR_INVALID_ARG
    assert f(8, 128, 64, 64, 0, 0, 0, out) == _abi.MOE_ERR_INVALID_ARG
    for bad in ((0, 128, 64), (17, 128, 64), (8, 100, 64), (8, 128, 24)):
        assert f(*bad, 64, 0, 0, 148, out) == _abi.MOE_ERR_UNSUPPORTED
