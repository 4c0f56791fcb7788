"""Host code of the entry points when a CUDA call fails, on a stand-in for the CUDA runtime
(fake_runtime.cpp): whichever call fails, the entry point says so, gives its workspaces back,
and leaves no kernel on its side stream that the caller's stream does not wait for.  No GPU."""
import concurrent.futures
import ctypes
import os
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
P = ctypes.c_void_p(1 << 20)
STREAM = ctypes.c_void_p(0x7770)
OK, CUDA = 0, 4
ALLOC, FREE, LAUNCH, RECORD, WAIT, SYNC, OTHER = range(7)


@pytest.fixture(scope="module")
def objects(tmp_path_factory):
    """The library linked with the stand-in (kernels as PTX only: none is run)."""
    from gqa_attention_flash_b200 import build
    out = tmp_path_factory.mktemp("fake")

    def compile_one(src):
        obj = str(out / (os.path.basename(src) + ".o"))
        subprocess.run([build.nvcc(), "-gencode", "arch=compute_100a,code=compute_100a", "-std=c++17", "-c",
                        "-Xcompiler", "-fPIC", "-I", build.INCLUDE, "-I", build.CSRC, src, "-o", obj],
                       check=True)
        return obj

    with concurrent.futures.ThreadPoolExecutor(8) as pool:
        objs = list(pool.map(compile_one, [*build.sources(), os.path.join(HERE, "fake_runtime.cpp")]))
    return out, objs


def fresh(objects):
    """A copy of the library of its own: what it makes once (streams, pools) is not made yet."""
    out, objs = objects
    lib = str(out / f"lib{len(os.listdir(out))}.so")
    subprocess.run(["g++", "-shared", "-Wl,-Bsymbolic", "-o", lib, *objs, "-ldl", "-lpthread"], check=True)
    lib = ctypes.CDLL(lib)
    lib.fake_log.argtypes = [ctypes.c_int] + [ctypes.c_void_p] * 3
    return lib


def log(lib):
    k, s, w = ctypes.c_int(), ctypes.c_void_p(), ctypes.c_void_p()
    for i in range(lib.fake_log_size()):
        lib.fake_log(i, ctypes.byref(k), ctypes.byref(s), ctypes.byref(w))
        yield k.value, s.value, w.value


def check_log(lib, where):
    live, side, recorded = set(), {}, {}
    for kind, stream, what in log(lib):
        if kind == ALLOC:
            live.add(what)
        elif kind == FREE:
            assert what in live, where
            assert not side, f"{where}: a workspace is freed while a side stream may use it"
            live.discard(what)
        elif kind == LAUNCH and stream != STREAM.value:
            side[stream] = True
        elif kind == RECORD:
            recorded[what] = stream
        elif kind == WAIT and stream == STREAM.value:
            side.pop(recorded.get(what), None)
        elif kind == SYNC:
            side.pop(stream, None)
    assert not live, f"{where}: {len(live)} workspaces are not given back"
    assert not side, f"{where}: a side stream is not joined"


def f(x):
    return ctypes.c_float(x)


def backward(B, Hq, Hkv, S, D, window, sinks):
    def call(L):
        return L.attn_bwd_sinks(P, P, P, P, P, P, P, P, P, B, Hq, Hkv, S, S, D, f(0.1), window, sinks, 0,
                                None, None, STREAM)
    return call


CALLS = {
    "backward, two streams": backward(4, 32, 8, 4096, 128, 1024, 4),
    "backward, two streams, split": backward(1, 32, 1, 1300, 64, 64, 4),
    "backward, one stream, split": backward(2, 8, 2, 1000, 64, 200, 5),
    "backward, plain": lambda L: L.attn_bwd(P, P, P, P, P, P, P, P, P, 1, 8, 2, 2048, 2048, 128, f(0.1), 1, 0,
                                            0, None, None, STREAM),
    "forward": lambda L: L.attn_fwd_sinks(P, P, P, P, P, 1, 8, 2, 300, 300, 128, f(0.1), 64, 4, 0, None, None,
                                          STREAM),
    "decode": lambda L: L.attn_decode_sinks(P, P, P, P, P, 64, 4, 4, STREAM, 2, 8, 2, 512, 128),
    "decode, workspace": lambda L: L.attn_decode_sinks(P, P, P, P, P, 64, 4, 16, STREAM, 2, 8, 2, 512, 128),
    "decode, slices chosen": lambda L: L.attn_decode_sinks(P, P, P, P, P, 64, 4, 0, STREAM, 2, 8, 2, 512, 128),
    "paged decode, slices chosen": lambda L: L.attn_decode_paged_sinks(P, P, P, P, P, P, 64, 4, 0, STREAM, 2, 8, 2,
                                                                       9, 16, 4, 128),
    "paged decode": lambda L: L.attn_decode_paged_sinks(P, P, P, P, P, P, 64, 4, 16, STREAM, 2, 8, 2, 9, 16, 4,
                                                        128),
    "tree": lambda L: L.attn_tree_paged(P, P, P, P, P, P, P, None, STREAM, 2, 8, 2, 5, 9, 16, 4, 128),
    "append": lambda L: L.attn_cache_append(P, P, P, P, P, P, None, STREAM, 2, 2, 5, 9, 16, 4, 128),
    "compact": lambda L: L.attn_cache_compact(P, P, P, P, P, None, STREAM, 2, 2, 5, 9, 16, 4, 128),
    "copy_blocks": lambda L: L.attn_cache_copy_blocks(P, P, P, P, STREAM, 3, 9, 16, 2, 128),
    "fork": lambda L: L.attn_cache_fork(P, P, P, P, P, P, P, STREAM, 3, 4, 9, 16, 4),
    "extend": lambda L: L.attn_cache_extend(P, P, P, P, STREAM, 4, 9, 16, 4),
    "free": lambda L: L.attn_cache_free(P, P, P, P, P, STREAM, 3, 4, 9, 4),
}


@pytest.mark.parametrize("name", CALLS)
def test_a_failing_cuda_call(objects, name):
    call = CALLS[name]
    lib = fresh(objects)
    lib.fake_reset(-1)
    assert call(lib) == OK
    check_log(lib, name)
    first = lib.fake_calls()
    for warm in (False, True):  # on the first call of a process, and on a later one
        for at in range(first):
            lib = fresh(objects) if not warm else lib
            lib.fake_reset(at)
            rc = call(lib)
            if lib.fake_calls() <= at:
                assert warm and rc == OK  # fewer calls once the set-up is done
                break
            assert rc == CUDA, f"{name}: call {at} of {first} fails, and the answer is {rc}"
            check_log(lib, f"{name}: call {at} of {first} fails")
            # the runtime's last error is clean again, for this library's calls and any other's
            assert lib.fake_last_error() == 0, f"{name}: call {at} of {first} fails"


@pytest.mark.parametrize("name", CALLS)
def test_an_error_of_other_code_is_not_the_calls(objects, name):
    """An error that the process left with the runtime before the call is neither reported nor
    cleared by it."""
    lib = fresh(objects)
    lib.fake_reset(-1)
    lib.fake_set_last_error(2)
    assert CALLS[name](lib) == OK
    assert lib.fake_last_error() == 2


def test_slices_of_the_windowed_decode_follow_the_devices_sms(objects):
    lib = fresh(objects)
    lib.fake_reset(-1)
    # two (sequence, KV head) pairs, 512 key tiles: two blocks for each SM
    for sms, slices in ((148, 64), (8, 8), (6, 6), (1, 1)):
        lib.fake_set_sms(sms)
        assert lib.attn_decode_sinks(P, P, P, P, P, 1 << 15, 4, 0, STREAM, 1, 8, 2, 1 << 15, 128) == OK
        if slices > 8:  # the combine came last, 8 heads in blocks of 4
            assert lib.fake_last_grid_x() == 2
        else:
            assert lib.fake_last_grid_x() == slices
